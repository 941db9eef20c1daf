// moe_mm.hip -- products over ragged groups of rows with ROW-MAJOR operands:
// 16-bit (bf16, fp16) forward product and both gradients, and the int8
// product with one scale per token and per channel.
//
// Every product is D[m][n] = sum_k P(m, k) Q(n, k) on 256-column tiles of
// BM output rows.  An operand is either "C" (k runs along its memory rows:
// x, w forward, dy in kDgrad) or "T" (k is the row index: w in kDgrad, both
// operands of kWgrad).  A K step is 128 bytes of every C row (64 16-bit or
// 128 int8 values) or 64 rows of a T operand, brought by direct-to-LDS
// loads into one stage of a ring while another is multiplied.
//   C stage: rows of 128 bytes, 16-byte chunk c of row r at slot c ^ (r & 7),
//     so that the 16 lanes that read one chunk of 16 rows for the MFMA spread
//     over the banks while a load still covers whole 128-byte lines.
//   T stage: 64 rows of 2 W bytes; the 32-byte granule q (16 columns) of row
//     r at slot q ^ f(r), f from bits 0, 1, 3, 4 of r: the transposing LDS
//     read takes 4 rows x 16 columns per 16 lanes, rows 8 g + 0..3 for the
//     wave's four lane groups, and f sends those 16 rows to 16 granules.
// Rows, columns and K steps past an operand's end read zeros through the
// buffer descriptor's bounds check, which ends at the group's last row, so a
// NaN of another group never meets this one's zeros.
//
// Large products are bound by the loads' way into LDS together with the power
// that the matrix units draw: one 4096 x 4096 x 7168 bf16 product takes 170 us
// (1416 TFLOP/s; the library's 156 us on the same card, but dx 186 against 189
// and dW 182 against 224), 70 % of the cycles in MFMAs at 1.9 GHz; without
// loads 155 us, without MFMAs 122, and on zeros, which draw less, 156.  Ragged
// groups of cold weights wait for HBM on top of it (E=64, 32768 rows, 4096 ->
// 1536: 440 us, 936 TFLOP/s).
#include <cmath>

#include "moe_device.h"
#include "moe_mm.h"
#include "moe_quant_i8.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));

constexpr int kThreads = 512;
constexpr int kBN = 256;     // output columns of a tile
constexpr double kCUs = 256;
constexpr int kStepRows = 64;  // k rows of a T stage
constexpr uint32_t kOutside = 0x80000000u;  // a byte offset no descriptor reaches

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
}

// Direct-to-LDS load of 16 bytes per lane: lane l's land at lds + 16 l (lds
// wave-uniform).  `off` counts from `base`; from `span` on it reads zeros.
// STREAM: read once, so not kept in the caches (non-temporal).
template <bool STREAM>
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t span, uint32_t off, uint8_t* lds) {
  auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, span, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0,
                                           STREAM ? 2 : 0);
}

// Barrier after this wave's LDS accesses and loads have completed; nothing is
// scheduled across it.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0), lgkmcnt(0)
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// The same, but for this wave's last N loads.
template <int N>
__device__ __forceinline__ void stage_barrier_but() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070 | (N & 15) | ((N >> 4) << 14));
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Barrier after this wave's LDS accesses; loads stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0xC07F);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// 16 bytes per lane to base + off, past the caches; nothing for kOutside.
__device__ __forceinline__ void store16(uint8_t* base, const v4i& v, uint32_t off) {
  auto r = __builtin_amdgcn_make_buffer_rsrc(base, 0, 0x7FFFFFFF, 0x00020000);
  __builtin_amdgcn_raw_buffer_store_b128(v, r, off, 0, 2);
}

// A group's rows and the tile's place in it.
struct Place {
  int e;      // group; E and E + 1: the rows behind the last and before the first one (clear_rest)
  int row0;   // first row of the tile
  int rows;   // rows of the tile (<= BM)
};

// Row range of group e (E: the rows behind the last group, E + 1: those before
// the first): the offsets clamped to [0, R], so a wrong offset array reads and
// writes nothing outside the tensors.
__device__ __forceinline__ int2 group_rows(const int32_t* offsets, int e, int E, int R) {
  if (!offsets) return make_int2(e ? R : 0, R);
  if (e > E) return make_int2(0, min(max(offsets[0], 0), R));
  const int a = min(max(offsets[e], 0), R);
  const int b = e < E ? min(max(offsets[e + 1], a), R) : R;
  return make_int2(a, b);
}

// Tile `t` of the launch: every wave scans the groups' tile counts (64 lanes
// at a time), so nothing has to be prepared on the host.  `id` runs over this
// launch's workgroups; workgroup ids are dealt round-robin over the 8 XCDs,
// and XCD x takes tiles [x per, (x + 1) per): neighbouring tiles, which share
// rows or weights, share an L2.  Tiles run over all columns of four row tiles
// before the next four, of eight where there are eight columns or more
// (measured with 6, 8 and 16 columns: 4 and 8 are within 2 % of the best of 2,
// 4, 8 and 16).  Returns false where the id has no tile.
__device__ __forceinline__ bool find_tile(const MmArgs& a, int BM, int ncol, int id, Place& pl, int& col) {
  const int lane = threadIdx.x & 63;
  const int G = a.E + (a.clear_rest ? 2 : 0);
  // inclusive scan of 64 groups' tile counts, from group e0 on
  int2 r;
  int n, incl;
  auto scan = [&](int e0) __attribute__((always_inline)) {
    n = 0;
    r = make_int2(0, 0);
    if (e0 + lane < G) {
      r = group_rows(a.offsets, e0 + lane, a.E, a.R);
      n = (r.y - r.x + BM - 1) / BM;
    }
    incl = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl = __builtin_elementwise_add_sat(incl, v);
    }
  };
  int total = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    scan(e0);
    total = __builtin_elementwise_add_sat(total, __builtin_amdgcn_readlane(incl, 63));
  }
  // A launch has fewer than 2^24 tiles (see plan).  Offsets that decrease can name
  // rows many times over, and their tiles pass 32 bits: then there is none.
  if (uint64_t(uint32_t(total)) * uint32_t(ncol) >= 0x7FFFFFFFu) return false;
  const uint32_t tiles = uint32_t(total) * uint32_t(ncol), per = (tiles + 7) / 8;
  const uint32_t t = (id & 7) * per + (id >> 3);
  if (uint32_t(id >> 3) >= per || t >= tiles) return false;
  const uint32_t high = ncol < 8 ? 4 : 8;
  const uint32_t block = t / (high * ncol), in = t - block * high * ncol;
  const uint32_t wide = min(high, uint32_t(total) - block * high);  // row tiles of this block of columns
  col = int(in / wide);
  const int want = int(block * high + in % wide);
  int before = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    if (G > 64) scan(e0);  // else as it stands
    const uint64_t past = __ballot(before + incl > want);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = before + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(n, l);
      pl.e = e0 + l;
      pl.row0 = __builtin_amdgcn_readlane(r.x, l) + (want - first) * BM;
      pl.rows = min(BM, __builtin_amdgcn_readlane(r.y, l) - pl.row0);
      return true;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

template <int TY> struct Acc { typedef v4f type; };
template <> struct Acc<kInt8> { typedef v4i type; };

template <int TY>
__device__ __forceinline__ typename Acc<TY>::type mma(const v4i& a, const v4i& b, const typename Acc<TY>::type& c) {
  if constexpr (TY == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
  else if constexpr (TY == kFp16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, a), __builtin_bit_cast(h8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// four fp32 results in a 16-bit type, rounded once (to nearest even; NaN and
// infinity stay)
__device__ __forceinline__ uint2 round4(const v4f& v, int ty) {
  typedef _Float16 h4 __attribute__((ext_vector_type(4)));
  typedef __bf16 b4 __attribute__((ext_vector_type(4)));
  return ty == kFp16 ? __builtin_bit_cast(uint2, __builtin_convertvector(v, h4))
                     : __builtin_bit_cast(uint2, __builtin_convertvector(v, b4));
}
__device__ __forceinline__ void store4(void* out, long at, const v4f& v, int ty) {
  if (ty == kFp32) *reinterpret_cast<v4f*>(static_cast<float*>(out) + at) = v;
  else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = round4(v, ty);
}

// The result of a sum: itself, or for int8 (sum * token's scale) * channel's
// scales (in fp32).  Rows of no group, and rows that name no token, are zeros.
template <int TY>
__device__ __forceinline__ v4f scaled(const MmArgs& a, int e, int row, int c, const typename Acc<TY>::type& sum) {
  if constexpr (TY == kInt8) {
    if (e >= a.E) return v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const int t = a.row_token ? a.row_token[row] : row;
    if (a.row_token && (t < 0 || t >= a.T)) return v4f{0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_convertvector(sum, v4f) * a.ps[t] * *reinterpret_cast<const v4f*>(a.qs + long(e) * a.N + c);
  } else {
    return sum;
  }
}

// The stream of one operand's tile over the K steps: ROWS rows of a C
// operand, or 64 rows of ROWS columns of a T operand per step.  The base
// moves along with the steps, so the descriptor's 32-bit range only has to
// span one tile.
template <bool TR, int ROWS>
struct Stream {
  static constexpr int kBytes = TR ? kStepRows * ROWS * 2 : ROWS * 128;
  static constexpr int kLoads = kBytes / 1024 / 8;  // 1 KB wave loads per wave
  const uint8_t* base;
  long left;       // bytes from base to the end of what may be read
  long step;       // bytes per K step
  uint32_t off[kLoads];
  int chunk;       // C: byte of the lane's chunk in the 128-byte step

  // `b`: the first byte; `bytes` may be read from there on; `ld`: bytes per memory
  // row.  `index` (C): the memory row of each of the tile's nindex rows, counted
  // from b; one outside [0, nrows_of_p) reads as zeros.
  __device__ __forceinline__ void init(const uint8_t* b, long bytes, long ld, int w, int lane,
                                       const int32_t* index, int nindex, int nrows_of_p) {
    base = b;
    left = bytes;
    step = TR ? kStepRows * ld : 128;
    chunk = TR ? 0 : ((lane & 7) ^ (lane >> 3)) * 16;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = w * kLoads + i;  // the load's kilobyte of the stage
      if constexpr (TR) {
        constexpr int kPerRow = ROWS * 2 / 16;  // 16-byte slots per row
        const int slot = at * 64 + lane, row = slot / kPerRow, s = slot % kPerRow;
        const int f = ((row & 3) | ((row >> 3) & 3) << 2) & (ROWS / 16 - 1);
        off[i] = uint32_t(row * ld) + (((s >> 1) ^ f) * 32 + (s & 1) * 16);
      } else {
        const int row = at * 8 + (lane >> 3);
        if (index) {
          const int t = row < nindex ? index[row] : -1;
          off[i] = t >= 0 && t < nrows_of_p ? uint32_t(t * ld) + chunk : kOutside;
        } else {
          off[i] = uint32_t(row * ld) + chunk;
        }
      }
    }
  }

  // Issue one step's loads into `stage`.  kleft: C: valid bytes of this step
  // (a multiple of 16; chunks past them read as zeros).
  __device__ __forceinline__ void issue(uint8_t* stage, int w, int kleft) const {
    const uint32_t n = uint32_t(left < 0 ? 0L : left > 0x7FFFFFFFL ? 0x7FFFFFFFL : left);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      dma16<false>(base, n, TR || chunk < kleft ? off[i] : kOutside, stage + (w * kLoads + i) * 1024);
  }
  __device__ __forceinline__ void advance() {
    base += step;
    left -= step;
  }
};

// MFMA fragment `frag` (16 rows or columns) of a stage for this lane; kk: the
// half of the K step.
template <bool TR, int ROWS>
__device__ __forceinline__ v4i read_frag(const uint8_t* stage, int frag, int kk, int lane) {
  const int m = lane & 15, g = lane >> 4;
  if constexpr (TR) {
    const int row = kk * 32 + 8 * g + (m >> 2);
    const int f = ((m >> 2) | g << 2) & (ROWS / 16 - 1);
    const uint8_t* at = stage + row * (ROWS * 2) + ((frag ^ f) * 32) + (m & 3) * 8;
    const s4v lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(at));
    const s4v hi =
        __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s4v*)(at + 4 * ROWS * 2));
    const int2 l = __builtin_bit_cast(int2, lo), h = __builtin_bit_cast(int2, hi);
    return v4i{l.x, l.y, h.x, h.y};
  } else {
    return *reinterpret_cast<const v4i*>(stage + (frag * 16 + m) * 128 + (((kk * 4 + g) ^ (m & 7)) << 4));
  }
}

// Tiles of the weight gradient that an XCD takes in a run, of `one` in a group
// and `total` of all.  Groups differ in length, so it is an eighth of a group's;
// where every workgroup has one tile, it is an eighth of all.
__host__ __device__ constexpr long run_of(long one, long total) { return ((total <= long(kCUs) ? total : one) + 7) / 8; }

template <int OP, int TY, int BM, bool kTurns = false>
__global__ __launch_bounds__(kThreads) void k_mm(MmArgs a) {
  constexpr bool PT = OP == kWgrad, QT = OP != kFwd;
  constexpr int NF = 4;             // column fragments of a wave (64 columns)
  constexpr int MF = BM / 32;       // row fragments of a wave (BM / 2 rows)
  constexpr int kEl = TY == kInt8 ? 1 : 2;
  constexpr int kStep = 128 / kEl;  // reduction length of a step
  using PS = Stream<PT, BM>;
  using QS = Stream<QT, kBN>;
  // Stages: as many as the CU's LDS holds (two workgroups of BM = 64 share it).
  // Each is needed a step later than its loads go out, so a third one gives
  // loads that miss the L2 two steps' time.  (Cold operands, us, two stages of both and
  // these: ragged groups, 32768 rows, 4096 -> 1536, E=64, forward 470 and 435, dx 484 and
  // 456; 12248 rows, 2048 -> 1408, E=64, forward 123 and 117, dx 158 and 129; dW of 16
  // groups of 1024, 2048 -> 4096, 299 and 266 to 279; nothing where all is in the L2.)
  // kTurns: a workgroup takes several tiles of dW in turn, and the next one's first
  // stages load while one is stored from pieces of LDS of its own, which take
  // the third stage's place (see takes_turns).
  constexpr int NP = BM == 128 ? 3 : 2, NQ = BM == 64 || kTurns ? 2 : 3;
  // one array per stage: the compiler's alias analysis then keeps a stage's
  // reads free of waits for the other stage's loads
  __shared__ __align__(1024) uint8_t p0[PS::kBytes];
  __shared__ __align__(1024) uint8_t p1[PS::kBytes];
  __shared__ __align__(1024) uint8_t p2[NP > 2 ? PS::kBytes : 16];
  __shared__ __align__(1024) uint8_t q0[QS::kBytes];
  __shared__ __align__(1024) uint8_t q1[QS::kBytes];
  __shared__ __align__(1024) uint8_t q2[NQ > 2 ? QS::kBytes : 16];
  __shared__ __align__(1024) uint8_t pieces[kTurns ? kThreads / 64 * 2048 : 16];

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 2, wn = w & 3;
  const int cols = OP == kFwd ? a.N : a.K;  // output columns
  const int ncol = (cols + kBN - 1) / kBN;

  Place pl;
  int ct, red = 0, split = 0;  // column tile, reduction length, share of the group's rows
  PS ps;
  QS qs;
  const uint8_t* P = static_cast<const uint8_t*>(a.p);
  const uint8_t* Q = static_cast<const uint8_t*>(a.q);
  // kWgrad: tile of group e: rows are N, columns K.  All tiles have one number
  // (group, share of its rows, column, row: those of a column share its strip of
  // x), and runs of them are dealt to the XCDs.  A group's rows may be split over
  // a.splits workgroups, in whole steps.
  // turn: the tile's number on this XCD; false behind the last one.
  auto place_wgrad = [&](uint32_t turn) __attribute__((always_inline)) {
    const uint32_t nrow = (a.N + BM - 1) / BM, one = nrow * ncol, total = one * a.E * a.splits;
    const uint32_t run = run_of(one, total);
    const uint32_t f = (turn / run * 8 + (blockIdx.x & 7)) * run + turn % run;
    // (the last runs of an XCD may lie behind the end: so do all its turns from there on)
    if (f >= total) return false;
    const uint32_t part = f / one, in = f - part * one;
    pl.e = int(part / a.splits);
    split = int(part - pl.e * uint32_t(a.splits));
    ct = int(in / nrow);
    pl.row0 = int(in % nrow) * BM;
    pl.rows = min(BM, a.N - pl.row0);
    const int2 r = group_rows(a.offsets, pl.e, a.E, a.R);
    const int all = r.y - r.x, each = ((all + kStep - 1) / kStep + a.splits - 1) / a.splits * kStep;
    const int skip = int(min(long(split) * each, long(all)));
    const int ra = __builtin_amdgcn_readfirstlane(r.x + skip);
    red = __builtin_amdgcn_readfirstlane(min(each, all - skip));
    ps.init(P + (long(ra) * a.N + pl.row0) * 2, (long(red) * a.N - pl.row0) * 2, long(a.N) * 2, w, lane, nullptr, 0, 0);
    qs.init(Q + (long(ra) * a.K + ct * kBN) * 2, (long(red) * a.K - ct * kBN) * 2, long(a.K) * 2, w, lane, nullptr, 0,
            0);
    return true;
  };
  uint32_t turn = blockIdx.x >> 3;
  if constexpr (OP == kWgrad) {
    if (!place_wgrad(turn)) return;
  } else {
    if (!find_tile(a, BM, ncol, blockIdx.x, pl, ct)) return;
    red = OP == kFwd ? a.K : a.N;
    const long ldp = long(red) * kEl;  // bytes per row of p
    if (a.row_token)
      ps.init(P, long(a.T) * ldp, ldp, w, lane, a.row_token + pl.row0, pl.rows, a.T);
    else
      ps.init(P + pl.row0 * ldp, pl.rows * ldp, ldp, w, lane, nullptr, 0, 0);
    const uint8_t* we = Q + long(pl.e) * a.N * a.K * kEl;
    if constexpr (OP == kFwd)
      qs.init(we + long(ct) * kBN * ldp, long(min(kBN, a.N - ct * kBN)) * ldp, ldp, w, lane, nullptr, 0, 0);
    else
      qs.init(we + ct * kBN * 2, (long(a.N) * a.K - ct * kBN) * 2, long(a.K) * 2, w, lane, nullptr, 0, 0);
    if (pl.e >= a.E) {  // rows of no group: zeros
      red = 0;
      qs.left = 0;
    }
  }
  typename Acc<TY>::type acc[MF][NF];
  int kleft_p = OP == kWgrad ? 0 : red * kEl, kleft_q = kleft_p;  // bytes of a C row from the next step to load on
  auto issue_p = [&](uint8_t* sp) __attribute__((always_inline)) {
    ps.issue(sp, w, kleft_p);
    ps.advance();
    kleft_p -= 128;
  };
  auto issue_q = [&](uint8_t* sq) __attribute__((always_inline)) {
    qs.issue(sq, w, kleft_q);
    qs.advance();
    kleft_q -= 128;
  };
  // The fragments of half a step.  Each half is read while the half before it
  // is multiplied, so a step has one barrier, between its halves: by then every
  // wave has read the whole stage, whose place the next loads take, and the next
  // stage has arrived.  Loads complete in the order they went out, so it is enough
  // to wait for all but those of the stages after that one.
  struct Half {
    v4i p[MF], q[NF];
  };
  auto read = [&](Half& f, const uint8_t* sp, const uint8_t* sq, int kk) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < NF; ++j) f.q[j] = read_frag<QT, kBN>(sq, wn * NF + j, kk, lane);
#pragma unroll
    for (int i = 0; i < MF; ++i) f.p[i] = read_frag<PT, BM>(sp, wm * MF + i, kk, lane);
  };
  auto multiply = [&](const Half& f) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = mma<TY>(f.q[j], f.p[i], acc[i][j]);
  };
  Half even, odd;
  // one step from stage x, with y the next stage (what is read from it after
  // the last step goes unused)
  auto step = [&](uint8_t* px, uint8_t* qx, const uint8_t* py, const uint8_t* qy) __attribute__((always_inline)) {
    read(odd, px, qx, 1);
    multiply(even);
    stage_barrier_but<(NP - 2) * PS::kLoads + (NQ - 2) * QS::kLoads>();  // the next stage has arrived
    issue_p(px);
    issue_q(qx);
    read(even, py, qy, 0);
    multiply(odd);
#pragma unroll
    for (int i = 0; i < PS::kLoads + QS::kLoads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, MF * NF / 8, 0);
    }
  };
  auto start = [&]() __attribute__((always_inline)) {
    // in the order of the steps: p(s), q(s + NQ - 2), p(s + 1), ... (see step)
    issue_p(p0);
    issue_q(q0);
    if constexpr (NQ > NP) issue_q(q1);
    issue_p(p1);
    issue_q(NQ > NP ? q2 : q1);
    if constexpr (NP > 2) {
      issue_p(p2);
      issue_q(q2);
    }
  };
  // 16-bit stores of a wave and tile: two per 16 rows (fp32: twice as many)
  constexpr int kStores = 2 * MF;
  constexpr int kAhead = (NP - 1) * PS::kLoads + (NQ - 1) * QS::kLoads;
  static_assert(kAhead + kStores < 64, "vmcnt range");
  start();
  bool stored = false;  // the tile before is still being stored, in kStores stores
  for (;;) {
    // the first stage has arrived: all but the other stages' loads, and the
    // stores behind them, are complete
    if (kTurns && stored) stage_barrier_but<kAhead + kStores>();
    else stage_barrier_but<kAhead>();
    const int steps = (red + kStep - 1) / kStep;
#pragma unroll
    for (int i = 0; i < MF; ++i)
#pragma unroll
      for (int j = 0; j < NF; ++j) acc[i][j] = typename Acc<TY>::type{0, 0, 0, 0};
    read(even, p0, q0, 0);
    int s = 0;
    if constexpr (NQ == 2) {
      for (; s + 1 < steps; s += 2) {
        step(p0, q0, p1, q1);
        step(p1, q1, p0, q0);
      }
      if (s < steps) step(p0, q0, p1, q1);
    } else if constexpr (NP == 3) {
      for (; s + 2 < steps; s += 3) {
        step(p0, q0, p1, q1);
        step(p1, q1, p2, q2);
        step(p2, q2, p0, q0);
      }
      if (s < steps) {
        step(p0, q0, p1, q1);
        if (s + 1 < steps) step(p1, q1, p2, q2);
      }
    } else {
      for (; s + 5 < steps; s += 6) {
        step(p0, q0, p1, q1);
        step(p1, q1, p0, q2);
        step(p0, q2, p1, q0);
        step(p1, q0, p0, q1);
        step(p0, q1, p1, q2);
        step(p1, q2, p0, q0);
      }
      if (s < steps) {
        step(p0, q0, p1, q1);
        if (s + 1 < steps) {
          step(p1, q1, p0, q2);
          if (s + 2 < steps) {
            step(p0, q2, p1, q0);
            if (s + 3 < steps) {
              step(p1, q0, p0, q1);
              if (s + 4 < steps) step(p0, q1, p1, q2);
            }
          }
        }
      }
    }

    // Lane l holds columns 4 (l / 16) + 0..3 of row l % 16 of each fragment.
    // Sixteen rows at a time go through a piece of LDS of the wave's own, so that
    // a store covers whole rows of its 64 columns (128 or 256 bytes in a line)
    // instead of 32-byte pieces, and past the caches (268 MB of bf16 gradients, 16
    // groups of 1024 rows: 90 us less than in pieces).
    stage_barrier();  // no stage is read or filled any more
    const Place done = pl;
    const int done_ct = ct, done_split = split;
    bool more = false;
    if constexpr (kTurns) {
      turn += gridDim.x >> 3;
      more = place_wgrad(turn);
      if (more) start();
    }
    int el = lane;
    asm volatile("" : "+v"(el));  // addresses from here on are not formed before the loop, which has no registers for them
    const int m = el & 15, g = el >> 4;
    const long out_row0 = OP == kWgrad ? long(done.e) * a.N + done.row0 : long(done.row0);
    const int out_ty = OP == kWgrad && a.splits > 1 ? kFp32 : a.out_ty;
    void* out = OP == kWgrad && a.splits > 1 ? a.partial + long(done_split) * a.E * a.N * a.K : a.out;
    const int r0 = wm * (BM / 2), c0 = done_ct * kBN + wn * 16 * NF;
    uint8_t* rows0 = static_cast<uint8_t*>(out) + (out_row0 + r0) * cols * (out_ty == kFp32 ? 4 : 2);
#pragma unroll
    for (int i = 0; i < MF; ++i) {
      v4f v[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) {
        const int r = r0 + i * 16 + m, c = c0 + j * 16 + 4 * g;
        v[j] = TY == kInt8 && (r >= done.rows || c >= cols) ? v4f{0.0f, 0.0f, 0.0f, 0.0f}
                                                            : scaled<TY>(a, done.e, done.row0 + r, c, acc[i][j]);
      }
      uint8_t* piece = kTurns ? pieces + w * 2048 : (i & 1 ? q1 : q0) + w * 2048;
      // rows of 128 (256) bytes, their 16-byte chunks exchanged by the row's
      // number so that equal columns of different rows lie on different banks
      if (out_ty == kFp32) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {  // eight rows at a time
          if ((m >> 3) == u) {
#pragma unroll
            for (int j = 0; j < NF; ++j)
              *reinterpret_cast<v4f*>(piece + (m & 7) * 256 + (((4 * j + g) ^ (m & 7)) << 4)) = v[j];
          }
          __builtin_amdgcn_wave_barrier();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = h * 4 + (el >> 4), ch = el & 15;
            const v4i d = *reinterpret_cast<const v4i*>(piece + row * 256 + ((ch ^ row) << 4));
            const int r = i * 16 + u * 8 + row, c = c0 + ch * 4;
            store16(rows0, d, r0 + r < done.rows && c < cols ? uint32_t(r * cols + c) * 4 : kOutside);
          }
          __builtin_amdgcn_wave_barrier();
        }
      } else {
#pragma unroll
        for (int j = 0; j < NF; ++j)
          *reinterpret_cast<uint2*>(piece + m * 128 + (((2 * j + (g >> 1)) ^ (m & 7)) << 4) + (g & 1) * 8) =
              round4(v[j], out_ty);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = h * 8 + (el >> 3), ch = el & 7;
          const v4i d = *reinterpret_cast<const v4i*>(piece + row * 128 + ((ch ^ (row & 7)) << 4));
          const int r = i * 16 + row, c = c0 + ch * 8;
          store16(rows0, d, r0 + r < done.rows && c < cols ? uint32_t(r * cols + c) * 2 : kOutside);
        }
        __builtin_amdgcn_wave_barrier();
      }
    }
    if (!more) break;
    stored = out_ty != kFp32;
    if (!stored) wait_vm<0>();
  }
}

// The forward product where there are too few tiles for the chip (decoding, and
// dense products of up to a few hundred rows).  A workgroup makes 16 NC columns
// by 16 NT rows; each of its four waves takes a quarter of the K steps through
// a ring of S stages of its own, so nothing waits for another wave until the
// sums are added up, in the order of the waves, through LDS.  Bound by the
// weights' bytes and their latency: S - 1 steps of 2 KB per 16 columns are in
// flight per wave, on every CU.  One bf16 token through 8 of 64 experts, 4096 ->
// 1536: 18 us, 5.4 TB/s of weights; a stream of plain reads reaches 6.9 TB/s.
//
// S is 2, which lets the most workgroups share a CU's LDS.  With 2, 3 and 4
// stages, us, cold weights: 16 x 64 tiles (61 tokens, top-8 of 64, 1536 -> 4096) 130,
// 161, 174; 16 x 32 (6 matrices of 4096 x 4096, one int8 row each) 18, 20, 23; 32 x
// 16 (20000 rows in 8 groups, 4096 -> 16) 27, 28, 31; 32 x 32 (61 rows, 4096 -> 4096)
// 12.5, 13.9, 13.6; 32 x 64 (192 rows in 16 groups, 4096 -> 2048) 46, 48; 64 x 16 (612
// rows, 4096 -> 400) 13.0, 14.1, 13.7; 64 x 32 (1800 rows in 4 groups, 2048 -> 520)
// 24.2, 26.0.  16 x 16 tiles have four: as a rule they are what products of up to
// one tile per CU get, where nothing shares a CU and a deep ring hides the loads'
// latency (one row, 7168 -> 4096: 14.6, 12.1, 11.7; 8 groups of a row, three
// tiles per CU: 17.9, 18.4, 19.1).
constexpr int kFewWaves = 4;

template <int TY, int NC, int NT, int S>
__global__ __launch_bounds__(kFewWaves * 64) void k_mm_few(MmArgs a) {
  constexpr int kEl = TY == kInt8 ? 1 : 2;
  constexpr int L = 2 * (NC + NT);       // loads of a wave per step
  constexpr int kStage = L * 1024;       // bytes of a wave's stage
  typedef typename Acc<TY>::type acc_t;
  // one array per stage: see k_mm
  __shared__ __align__(1024) uint8_t st0[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st1[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st2[S == 4 ? kFewWaves * kStage : 16];
  __shared__ __align__(1024) uint8_t st3[S == 4 ? kFewWaves * kStage : 16];
  static_assert((S == 2 || S == 4) && (S - 1) * L < 64, "ring");
  static_assert(NC * NT * 1024 <= kStage, "a wave's sums fit a stage");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int ncol = (a.N + 16 * NC - 1) / (16 * NC);
  Place pl;
  int ct;
  if (!find_tile(a, 16 * NT, ncol, blockIdx.x, pl, ct)) return;
  const int ld = a.K * kEl;  // bytes per row of both operands
  const int n0 = ct * 16 * NC;
  const int steps = pl.e >= a.E ? 0 : (ld + 127) / 128;
  const int each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = w * each, mine = max(0, min(steps - s0, each));

  const uint8_t* wq = static_cast<const uint8_t*>(a.q) + (long(pl.e) * a.N + n0) * ld;
  const uint32_t wspan = uint32_t(min(16 * NC, a.N - n0)) * uint32_t(ld);
  const uint8_t* pq = static_cast<const uint8_t*>(a.p) + (a.row_token ? 0 : long(pl.row0) * ld);
  const uint32_t pspan = uint32_t(a.row_token ? a.T : pl.rows) * uint32_t(ld);
  // load i of a step covers rows 8 i .. 8 i + 7 of its operand; lane l has
  // row l / 8 and the 16-byte chunk that belongs in its slot l % 8
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t ow[2 * NC], op[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NC; ++i) ow[i] = uint32_t(8 * i + (lane >> 3)) * uint32_t(ld) + chunk;
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const int r = 8 * i + (lane >> 3);
    int t = r;
    if (a.row_token) {
      t = r < pl.rows ? a.row_token[pl.row0 + r] : -1;
      if (t >= a.T) t = -1;
    }
    op[i] = r < pl.rows && t >= 0 ? uint32_t(t) * uint32_t(ld) + chunk : kOutside;
  }

  acc_t acc[NC][NT];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = acc_t{0, 0, 0, 0};

  // step k of this wave; past its last one the loads read nothing, so that
  // every step has L loads for the waits to count
  auto issue = [&](uint8_t* stage, int k) __attribute__((always_inline)) {
    const int at = (s0 + k) * 128;
    const bool in = k < mine && chunk < ld - at;
    uint8_t* to = stage + w * kStage;
#pragma unroll
    for (int i = 0; i < 2 * NC; ++i) dma16<true>(wq, wspan, in ? ow[i] + at : kOutside, to + i * 1024);
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i)
      dma16<false>(pq, pspan, in && op[i] != kOutside ? op[i] + at : kOutside, to + (2 * NC + i) * 1024);
  };
  auto multiply = [&](const uint8_t* stage) __attribute__((always_inline)) {
    wait_vm<(S - 1) * L>();
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* sq = stage + w * kStage;
    const uint8_t* sp = sq + 2 * NC * 1024;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      v4i qf[NC], pf[NT];
#pragma unroll
      for (int i = 0; i < NC; ++i) qf[i] = read_frag<false, 16 * NC>(sq, i, kk, lane);
#pragma unroll
      for (int j = 0; j < NT; ++j) pf[j] = read_frag<false, 16 * NT>(sp, j, kk, lane);
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mma<TY>(qf[i], pf[j], acc[i][j]);
    }
    // the stage is read before its next loads go out
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  issue(st0, 0);
  if constexpr (S == 4) {
    issue(st1, 1);
    issue(st2, 2);
  }
  for (int k = 0; k < mine; k += S) {
    if constexpr (S == 2) {
      issue(st1, k + 1); multiply(st0);
      issue(st0, k + 2); multiply(st1);
    } else {
      issue(st3, k + 3); multiply(st0);
      issue(st0, k + 4); multiply(st1);
      issue(st1, k + 5); multiply(st2);
      issue(st2, k + 6); multiply(st3);
    }
  }

  stage_barrier();  // every load has landed: the first stage takes the sums
  acc_t* part = reinterpret_cast<acc_t*>(st0);
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(w * NC * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // fragment f's sum by wave f % 4: lane l holds columns 4 (l / 16) + 0..3 of row l % 16
  for (int f = w; f < NC * NT; f += kFewWaves) {
    acc_t sum = part[f * 64 + lane];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) sum += part[(v * NC * NT + f) * 64 + lane];
    const int r = (f % NT) * 16 + m, c = n0 + (f / NT) * 16 + 4 * g;
    if (r >= pl.rows || c >= a.N) continue;
    store4(a.out, (long(pl.row0) + r) * a.N + c, scaled<TY>(a, pl.e, pl.row0 + r, c, sum), a.out_ty);
  }
}

// moe_linear_i8 for one row: k_mm_few with the quantiser in front, in every
// workgroup: its lanes hold the row between the maximum and the rounding while
// the first weights are on their way; the codes stay in LDS, where all K steps
// read them.  Codes, sums and results are those of the two launches it stands
// for.  7168 -> 4096: 10.3 us as two launches, 7.9 as one (two rows this
// way: 12.2 against 11.0, so from there on it is two).
constexpr int kLinChunks = 4;  // chunks of 8 values that a lane keeps
constexpr int kLinMaxK = kLinChunks * kFewWaves * 64 * 8;

template <int XT, bool GLU, int NC>
__global__ __launch_bounds__(kFewWaves * 64) void k_linear_one(MmArgs a) {
  constexpr int S = 4, L = 2 * NC, kStage = L * 1024;
  __shared__ __align__(1024) uint8_t st0[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st1[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st2[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st3[kFewWaves * kStage];
  __shared__ __align__(16) uint8_t codes[kLinMaxK];
  __shared__ uint32_t s_top[kFewWaves];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int ncol = (a.N + 16 * NC - 1) / (16 * NC);
  Place pl;
  int ct;
  if (!find_tile(a, 16, ncol, blockIdx.x, pl, ct)) return;
  const int K = a.K, n0 = ct * 16 * NC;
  const bool grouped = pl.e < a.E;  // else the row belongs to no group: zeros
  const int steps = grouped ? (K + 127) / 128 : 0;
  const int each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = w * each, mine = max(0, min(steps - s0, each));
  const uint8_t* wq = static_cast<const uint8_t*>(a.q) + (long(pl.e) * a.N + n0) * K;
  const uint32_t wspan = uint32_t(min(16 * NC, a.N - n0)) * uint32_t(K);
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t ow[L];
#pragma unroll
  for (int i = 0; i < L; ++i) ow[i] = uint32_t(8 * i + (lane >> 3)) * uint32_t(K) + chunk;
  auto issue = [&](uint8_t* stage, int k) __attribute__((always_inline)) {
    const int at = (s0 + k) * 128;
    const bool in = k < mine && chunk < K - at;
#pragma unroll
    for (int i = 0; i < L; ++i) dma16<true>(wq, wspan, in ? ow[i] + at : kOutside, stage + w * kStage + i * 1024);
  };

  // the row comes in ahead of the first weights; one that names no token is zeros
  const int t = a.row_token ? a.row_token[pl.row0] : pl.row0;
  const bool token = grouped && (!a.row_token || (t >= 0 && t < a.T));
  const uint16_t* x = static_cast<const uint16_t*>(a.p) + long(token ? t : 0) * (GLU ? 2L * K : K);
  quant_raw8 raw[kLinChunks][GLU ? 2 : 1];
#pragma unroll
  for (int i = 0; i < kLinChunks; ++i) {
    const int c = (i * kFewWaves * 64 + int(threadIdx.x)) * 8;
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h)
      raw[i][h] = token && c < K ? *reinterpret_cast<const quant_raw8*>(x + h * K + c) : quant_raw8{0, 0, 0, 0};
  }
  __builtin_amdgcn_sched_barrier(0);
  issue(st0, 0);
  issue(st1, 1);
  issue(st2, 2);
  __builtin_amdgcn_sched_barrier(0);
  f8v v[kLinChunks];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kLinChunks; ++i) {
    v[i] = quant_value8<XT, GLU>(raw[i][0], raw[i][GLU ? 1 : 0]);
    top = max(top, quant_top8(v[i]));
  }
  for (int d = 1; d < 64; d <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, 64)));
  if (lane == 0) s_top[w] = top;
  lds_barrier();
  const QuantScale q = quant_scale(max(max(s_top[0], s_top[1]), max(s_top[2], s_top[3])));
#pragma unroll
  for (int i = 0; i < kLinChunks; ++i) {
    const int c = (i * kFewWaves * 64 + int(threadIdx.x)) * 8;
    // the last step's columns past K are zeros
    if (c < (K + 127) / 128 * 128) *reinterpret_cast<uint2*>(codes + c) = quant_codes8(v[i], q);
  }
  lds_barrier();

  v4i acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) acc[i] = v4i{0, 0, 0, 0};
  auto multiply = [&](const uint8_t* stage, int k) __attribute__((always_inline)) {
    wait_vm<(S - 1) * L>();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      v4i pf = {0, 0, 0, 0};
      if (m == 0 && k < mine) pf = *reinterpret_cast<const v4i*>(codes + (s0 + k) * 128 + (kk * 4 + g) * 16);
#pragma unroll
      for (int i = 0; i < NC; ++i)
        acc[i] = mma<kInt8>(read_frag<false, 16 * NC>(stage + w * kStage, i, kk, lane), pf, acc[i]);
    }
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int k = 0; k < mine; k += S) {
    issue(st3, k + 3); multiply(st0, k);
    issue(st0, k + 4); multiply(st1, k + 1);
    issue(st1, k + 5); multiply(st2, k + 2);
    issue(st2, k + 6); multiply(st3, k + 3);
  }
  stage_barrier();  // every load has landed: the first stage takes the sums
  v4i* part = reinterpret_cast<v4i*>(st0);
#pragma unroll
  for (int i = 0; i < NC; ++i) part[(w * NC + i) * 64 + lane] = acc[i];
  __syncthreads();
  if (w < NC && m == 0) {  // fragment w: lane l holds columns 4 (l / 16) + 0..3 of row l % 16
    v4i sum = part[w * 64 + lane];
#pragma unroll
    for (int u = 1; u < kFewWaves; ++u) sum += part[(u * NC + w) * 64 + lane];
    const int c = n0 + w * 16 + 4 * g;
    if (c < a.N) {
      v4f y = {0.0f, 0.0f, 0.0f, 0.0f};
      if (token)
        y = __builtin_convertvector(sum, v4f) * q.scale * *reinterpret_cast<const v4f*>(a.qs + long(pl.e) * a.N + c);
      store4(a.out, long(pl.row0) * a.N + c, y, a.out_ty);
    }
  }
}

// dw = the splits' fp32 sums added up in their order.
__global__ __launch_bounds__(256) void k_join(const float* __restrict__ part, int splits, long n, void* out, int ty) {
  for (long i = (long(blockIdx.x) * 256 + threadIdx.x) * 4; i < n; i += long(gridDim.x) * 1024) {
    v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
    int s = 0;
    for (; s + 8 <= splits; s += 8) {  // eight loads in flight
      v4f v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = *reinterpret_cast<const v4f*>(part + (s + u) * n + i);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += v[u];
    }
    for (; s < splits; ++s) sum += *reinterpret_cast<const v4f*>(part + s * n + i);
    store4(out, i, sum, ty);
  }
}

// Row tiles of a launch: sum over non-empty groups (and the rows outside them) of ceil(n / rows) at most.
long row_tiles(const MmArgs& a, int rows) {
  const long G = (a.E < a.R ? a.E : a.R) + (a.clear_rest ? 2 : 0);
  const long most = (long(a.R) + G * (rows - 1)) / rows;
  return most < a.R ? most : a.R;
}

// The shape of a launch: rows and columns of a tile; few: k_mm_few.
struct TileShape {
  int few, rows, cols;
};

// The tile shape whose launch brings the fewest bytes through a CU: rounds of
// one tile per CU times (rows + columns) of a tile.  Times follow that count
// where tiles do not yet fill the chip (one bf16 matrix, K = N = 4096, us: 64
// rows in tiles of 16 x 64 14.9, 32 x 32 13.9, 64 x 64 22.0, 64 x 256 59; 1024
// rows in 32 x 32 125, 64 x 64 79, 64 x 256 64, 256 x 256 76), and from there on it
// prefers the large tiles, which the matrix units need (E=64, 4096 -> 1536:
// 6144 rows in 64 x 256 222, 128 x 256 175, 256 x 256 198; 32768 rows 633, 470,
// 440).  The row tiles of ragged groups are estimated: groups with a row, each
// half a tile more than its mean needs.  Among equals the first, so the smaller
// tiles and k_mm_few (8 tokens, top-8 of 64: 94 us against 125).
TileShape shape_of(int op, const MmArgs& a, double* cost_of = nullptr) {
  if (op == kWgrad) return {0, 256, kBN};
  static const TileShape shapes[] = {{1, 16, 64}, {1, 16, 32}, {1, 16, 16}, {1, 32, 32}, {1, 32, 64}, {1, 32, 16},
                                     {1, 64, 64}, {1, 64, 32}, {1, 64, 16}, {0, 64, kBN}, {0, 128, kBN}, {0, 256, kBN}};
  const double cols = op == kFwd ? a.N : a.K;
  const double groups = a.E * (1.0 - std::exp(-double(a.R) / a.E));  // that are touched
  const double mean = a.R / std::fmax(groups, 1.0);
  TileShape best = {0, 256, kBN};
  double least = 1e300;
  for (const TileShape& s : shapes) {
    if (s.few && op != kFwd) continue;
    const double need = mean / s.rows;
    const double rows = a.E == 1 ? std::ceil(a.R / double(s.rows)) : groups * std::fmax(1.0, need + 0.5);
    const double cost = std::ceil(std::ceil(rows) * std::ceil(cols / s.cols) / kCUs) * (s.rows + s.cols);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  if (cost_of) *cost_of = least;
  return best;
}

// Workgroups of a launch in the given shape.
long grid_of(int op, const MmArgs& a, const TileShape& s) {
  const long cols = op == kFwd ? a.N : a.K, ncol = (cols + s.cols - 1) / s.cols;
  if (op == kWgrad) {
    const long one = (a.N + s.rows - 1) / s.rows * ncol, total = one * a.E * a.splits;
    const long runs = 8 * run_of(one, total);  // one of each XCD
    return (total + runs - 1) / runs * runs;
  }
  return (row_tiles(a, s.rows) * ncol + 7) / 8 * 8;
}

// The shape and the workgroups of a launch; false where no launch holds them.
// shape_of takes narrow tiles for narrow products, whatever their rows (N = 8: 64
// x 16 tiles, 2^24 workgroups at 2^30 rows); past a launch's limit it is the
// largest ones.
bool plan(int op, const MmArgs& a, TileShape* s, long* grid) {
  *s = shape_of(op, a);
  *grid = grid_of(op, a, *s);
  if (*grid <= max_blocks(s->few ? kFewWaves * 64 : kThreads)) return true;
  *s = {0, 256, kBN};
  *grid = grid_of(op, a, *s);
  return *grid <= max_blocks(kThreads);
}

// Rows of a dense product's first launch.  Where the last few rows would make
// the large tiles go one more round, they go into a launch of their own, in the
// shape that suits them; a launch counts as much as bringing in kLaunchBytes.
// (int8, N = 4096, us in one launch and in two, by the bytes that two save, in KB: 4099
// rows, K = 7168, 3441: 159 and 100; 2051, 7168, 688: 77 and 61; 2051, 4096, 393: 50 and
// 41; 300, 4096, 262: 20 and 16; 1030, 7168, 229: 44 and 68; 523, 7168, 229: 48 and
// 46; 1030, 4096, 131: 29 and 42; 523, 1024, 33: 10 and 16.)
constexpr double kLaunchBytes = 250e3;
int first_rows(int op, const MmArgs& a) {
  if (op != kFwd || a.offsets || a.R <= 256) return a.R;
  double one, head, tail;
  const int el = a.ty == kInt8 ? 1 : 2;
  shape_of(op, a, &one);
  const int rows = a.R / 256 * 256;
  MmArgs h = a, t = a;
  h.R = rows;
  t.R = a.R - rows;
  if (!t.R) return a.R;
  shape_of(op, h, &head);
  shape_of(op, t, &tail);
  return head + tail + kLaunchBytes / (double(a.K) * el) < one ? rows : a.R;
}

// Workgroups that share a group's rows in kWgrad: as many as leave the chip one
// tile per CU, while each keeps eight steps of 64 rows.  Their fp32 sums meet
// in a workspace and are added up in order.  (One matrix of 512 x 512 from
// 32768 rows: 521 us unsplit, 41 split.)
int splits_of(const MmArgs& a) {
  const double tiles = double(a.E) * ((a.N + 255) / 256) * ((a.K + kBN - 1) / kBN);
  const double steps = a.R / 64.0 / a.E;
  return int(std::fmax(1.0, std::fmin(std::floor(kCUs / tiles), std::floor(steps / 8))));
}

}  // namespace

size_t wgrad_bytes(const MmArgs& a) {
  const int s = splits_of(a);
  return s > 1 ? size_t(s) * a.E * a.N * a.K * 4 : 0;
}

// kWgrad: whether a workgroup per CU takes the tiles in turn, rather than one
// workgroup per tile.  Turns hide a tile's first loads and its stores, which
// counts where reductions are short; but they cost the third stage, the last
// round's empty places cost their whole length, and long groups are not evened out.
// places: the launch's workgroups, as one per tile: the tiles and the empty
// places behind the last of each XCD.
// (Cold operands, us, turns and one per tile: 64 groups, 1408 x 2048, 12 tiles per CU,
// of 16 rows 79 and 91, 128 105 and 113, 256 144 and 152, 1024 410 and 384; 256 groups,
// 512 x 512, of 128 47 and 48, 192 63 and 60; 16 groups, 4096 x 2048, of 128 77 and 82, 1024
// 300 and 266; 64 groups, 768 x 768, 2.25 per CU, of 128 32 and 31, 512 66 and 64.)
static bool takes_turns(const MmArgs& a, long places) {
  const double rows = double(a.R) / (double(a.E) * a.splits), each = places / kCUs;
  return each > 1 && rows <= 128 && rows * (std::ceil(each) / each - 1) < 64;
}

#define MOE_MM(kernel, threads) hipLaunchKernelGGL((kernel), dim3(grid), dim3(threads), 0, st, a)

template <int OP, int TY>
static hipError_t launch_shape(const MmArgs& a, const TileShape& s, unsigned grid, hipStream_t st) {
  if constexpr (OP == kWgrad) {
    if (takes_turns(a, grid)) hipLaunchKernelGGL((k_mm<OP, TY, 256, true>), dim3(unsigned(kCUs)), dim3(kThreads), 0, st, a);
    else MOE_MM((k_mm<OP, TY, 256>), kThreads);
    if (a.splits > 1) {
      const long n = long(a.E) * a.N * a.K, blocks = (n + 1023) / 1024;
      hipLaunchKernelGGL(k_join, dim3(unsigned(blocks < 2048 ? blocks : 2048)), dim3(256), 0, st, a.partial, a.splits, n,
                         a.out, a.out_ty);
    }
  } else {
    if constexpr (OP == kFwd) {
      if (s.few) {
#define MOE_FEW(NT, NC) \
  case NT * 16 + NC: MOE_MM((k_mm_few<TY, NC, NT, NT * NC == 1 ? 4 : 2>), kFewWaves * 64); break;
        switch (s.rows + s.cols / 16) {
          MOE_FEW(1, 1) MOE_FEW(1, 2) MOE_FEW(1, 4)
          MOE_FEW(2, 1) MOE_FEW(2, 2) MOE_FEW(2, 4)
          MOE_FEW(4, 1) MOE_FEW(4, 2) MOE_FEW(4, 4)
        }
#undef MOE_FEW
        return hipGetLastError();
      }
    }
    if (s.rows == 256) MOE_MM((k_mm<OP, TY, 256>), kThreads);
    else if (s.rows == 128) MOE_MM((k_mm<OP, TY, 128>), kThreads);
    else MOE_MM((k_mm<OP, TY, 64>), kThreads);
  }
  return hipGetLastError();
}
#undef MOE_MM

static hipError_t launch_one(int op, const MmArgs& a, const TileShape& s, long grid, hipStream_t st) {
  if (grid == 0) return hipSuccess;
  const unsigned g = unsigned(grid);
  if (a.ty == kInt8) return launch_shape<kFwd, kInt8>(a, s, g, st);
  if (a.ty == kBf16)
    return op == kFwd ? launch_shape<kFwd, kBf16>(a, s, g, st)
                      : op == kDgrad ? launch_shape<kDgrad, kBf16>(a, s, g, st) : launch_shape<kWgrad, kBf16>(a, s, g, st);
  return op == kFwd ? launch_shape<kFwd, kFp16>(a, s, g, st)
                    : op == kDgrad ? launch_shape<kDgrad, kFp16>(a, s, g, st) : launch_shape<kWgrad, kFp16>(a, s, g, st);
}

bool mm_too_large(int op, const MmArgs& args) {
  MmArgs a = args;
  a.splits = op == kWgrad ? splits_of(a) : 1;
  TileShape s;
  long grid;
  return !plan(op, a, &s, &grid);
}

hipError_t launch_mm(int op, const MmArgs& args, hipStream_t st, bool* too_large) {
  MmArgs a = args;
  a.splits = op == kWgrad ? splits_of(a) : 1;
  TileShape s;
  long grid;
  *too_large = !plan(op, a, &s, &grid);
  if (*too_large) return hipSuccess;
  const int rows = first_rows(op, a);
  if (rows == a.R) return launch_one(op, a, s, grid, st);
  MmArgs head = a, tail = a;
  const long el = a.ty == kInt8 ? 1 : 2, out_el = a.out_ty == kFp32 ? 4 : 2;
  head.R = rows;
  tail.R = a.R - rows;
  tail.out = static_cast<uint8_t*>(a.out) + long(rows) * a.N * out_el;
  if (a.row_token) {
    tail.row_token = a.row_token + rows;
  } else {
    tail.p = static_cast<const uint8_t*>(a.p) + long(rows) * a.K * el;
    if (a.ps) tail.ps = a.ps + rows;
  }
  TileShape ts;
  long tail_grid;
  *too_large = !plan(op, head, &s, &grid) || !plan(op, tail, &ts, &tail_grid);
  if (*too_large) return hipSuccess;
  const hipError_t e = launch_one(op, head, s, grid, st);
  return e != hipSuccess ? e : launch_one(op, tail, ts, tail_grid, st);
}

bool linear_is_one_launch(int R, int K) { return R <= 1 && K <= kLinMaxK; }

hipError_t launch_linear_one(const MmArgs& a, int x_ty, int swiglu, hipStream_t st) {
  // columns per workgroup as shape_of would choose them
  int nc = 1;
  double least = 1e300;
  for (int c = 2; c >= 1; --c) {
    const double cost = std::ceil(std::ceil(a.N / (16.0 * c)) / kCUs) * (16 + 16 * c);
    if (cost < least) {
      least = cost;
      nc = c;
    }
  }
  const long tiles = long(a.R) * ((a.N + 16 * nc - 1) / (16 * nc));
  const unsigned grid = unsigned((tiles + 7) / 8 * 8);
  if (!grid) return hipSuccess;
#define MOE_LIN(XT, GLU, NC) \
  hipLaunchKernelGGL((k_linear_one<XT, GLU, NC>), dim3(grid), dim3(kFewWaves * 64), 0, st, a)
#define MOE_LIN_NC(XT, GLU)            \
  do {                                 \
    if (nc == 2) MOE_LIN(XT, GLU, 2);  \
    else MOE_LIN(XT, GLU, 1);          \
  } while (0)
  if (x_ty == kBf16) {
    if (swiglu) MOE_LIN_NC(kBf16, true);
    else MOE_LIN_NC(kBf16, false);
  } else {
    if (swiglu) MOE_LIN_NC(kFp16, true);
    else MOE_LIN_NC(kFp16, false);
  }
#undef MOE_LIN_NC
#undef MOE_LIN
  return hipGetLastError();
}

}  // namespace moe
