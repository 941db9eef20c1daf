// moe_mm.hip -- products over ragged groups of rows with ROW-MAJOR operands:
// 16-bit (bf16, fp16) forward product and both gradients, and the int8
// product with one scale per token and per channel.
//
// Every product is D[m][n] = sum_k P(m, k) Q(n, k) on 256-column tiles of
// BM output rows.  An operand is either "C" (k runs along its memory rows:
// x, w forward, dy in kDgrad) or "T" (k is the row index: w in kDgrad, both
// operands of kWgrad).  A K step is 128 bytes of every C row (64 16-bit or
// 128 int8 values) or 64 rows of a T operand, brought by direct-to-LDS
// loads into one of two stages while the other is multiplied.
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
#include "moe_device.h"
#include "moe_mm.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef short s4v __attribute__((ext_vector_type(4)));
typedef __bf16 bf8v __attribute__((ext_vector_type(8)));

constexpr int kThreads = 512;
constexpr int kBN = 256;     // output columns of a tile
constexpr int kStepRows = 64;  // k rows of a T stage
constexpr uint32_t kOutside = 0x80000000u;  // a byte offset no descriptor reaches

#define LDS_PTR(p) ((__attribute__((address_space(3))) void*)(p))

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt(0x0F70 | (N & 15) | ((N >> 4) << 14));
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

// A group's rows and the tile's place in it.
struct Place {
  int e;      // group; E: the rows behind the last group (clear_tail)
  int row0;   // first row of the tile
  int rows;   // rows of the tile (<= BM)
};

// Row range of group e: the offsets clamped to [0, R], so a wrong offset
// array reads and writes nothing outside the tensors.
__device__ __forceinline__ int2 group_rows(const int32_t* offsets, int e, int E, int R) {
  if (!offsets) return make_int2(e ? R : 0, R);
  const int a = min(max(offsets[e], 0), R);
  const int b = e < E ? min(max(offsets[e + 1], a), R) : R;
  return make_int2(a, b);
}

// Tile `t` of the launch: every wave scans the groups' tile counts (64 lanes
// at a time), so nothing has to be prepared on the host.  `id` runs over this
// launch's workgroups; workgroup ids are dealt round-robin over the 8 XCDs,
// and XCD x takes tiles [x per, (x + 1) per): neighbouring tiles, which share
// rows or weights, share an L2.  Tiles run over all columns of four row
// tiles before the next four.  Returns false where the id has no tile.
__device__ __forceinline__ bool find_tile(const MmArgs& a, int BM, int ncol, int id, Place& pl, int& col) {
  const int lane = threadIdx.x & 63;
  const int G = a.E + (a.clear_tail ? 1 : 0);
  int total = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    int n = 0;
    if (e0 + lane < G) {
      const int2 r = group_rows(a.offsets, e0 + lane, a.E, a.R);
      n = (r.y - r.x + BM - 1) / BM;
    }
    for (int d = 1; d < 64; d <<= 1) n += __shfl_xor(n, d, 64);
    total += n;
  }
  total = __builtin_amdgcn_readfirstlane(total);
  const long tiles = long(total) * ncol;
  const long per = (tiles + 7) / 8;
  const long t = (id & 7) * per + (id >> 3);
  if ((id >> 3) >= per || t >= tiles) return false;
  const long block = t / (4L * ncol);
  const int in = int(t - block * 4 * ncol);
  const int wide = int(min(4L, total - block * 4));  // row tiles of this block of columns
  col = in / wide;
  const int want = int(block * 4) + in % wide;
  int before = 0;
  for (int e0 = 0; e0 < G; e0 += 64) {
    int n = 0;
    int2 r = make_int2(0, 0);
    if (e0 + lane < G) {
      r = group_rows(a.offsets, e0 + lane, a.E, a.R);
      n = (r.y - r.x + BM - 1) / BM;
    }
    int incl = n;
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
    const uint64_t past = __ballot(before + incl > want);
    if (past) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = before + __shfl(incl - n, l, 64);
      const int x = __shfl(r.x, l, 64), y = __shfl(r.y, l, 64);
      pl.e = __builtin_amdgcn_readfirstlane(e0 + l);
      pl.row0 = __builtin_amdgcn_readfirstlane(x + (want - first) * BM);
      pl.rows = min(BM, __builtin_amdgcn_readfirstlane(y) - pl.row0);
      return true;
    }
    before += __shfl(incl, 63, 64);
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

// four fp32 results to the output type, rounded once (to nearest even; NaN
// and infinity stay)
__device__ __forceinline__ void store4(void* out, long at, const v4f& v, int ty) {
  if (ty == kFp32) {
    *reinterpret_cast<v4f*>(static_cast<float*>(out) + at) = v;
  } else if (ty == kFp16) {
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<h4*>(static_cast<_Float16*>(out) + at) = __builtin_convertvector(v, h4);
  } else {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<b4*>(static_cast<__bf16*>(out) + at) = __builtin_convertvector(v, b4);
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

  // `ld`: bytes per memory row.  rows: C: valid rows of the tile.
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
    auto r = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, n, 0x00020000);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t o = TR || chunk < kleft ? off[i] : kOutside;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(r, LDS_PTR(stage + (w * kLoads + i) * 1024), 16, o, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void advance() {
    base += step;
    left -= step;
  }
};

// MFMA fragment i (16 rows / columns) of a stage for this lane; kk: the half
// of the K step; t0: the first fragment of the wave in the stage.
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

template <int OP, int TY, int BM>
__global__ __launch_bounds__(kThreads) void k_mm(MmArgs a) {
  constexpr bool PT = OP == kWgrad, QT = OP != kFwd;
  constexpr int NF = 4;             // column fragments of a wave (64 columns)
  constexpr int MF = BM / 32;       // row fragments of a wave (BM / 2 rows)
  constexpr int kEl = TY == kInt8 ? 1 : 2;
  constexpr int kStep = 128 / kEl;  // reduction length of a step
  using PS = Stream<PT, BM>;
  using QS = Stream<QT, kBN>;
  // one array per stage: the compiler's alias analysis then keeps a stage's
  // reads free of waits for the other stage's loads
  __shared__ __align__(1024) uint8_t p0[PS::kBytes];
  __shared__ __align__(1024) uint8_t p1[PS::kBytes];
  __shared__ __align__(1024) uint8_t q0[QS::kBytes];
  __shared__ __align__(1024) uint8_t q1[QS::kBytes];

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 2, wn = w & 3;
  const int cols = OP == kFwd ? a.N : a.K;  // output columns
  const int ncol = (cols + kBN - 1) / kBN;

  Place pl;
  int ct, red;  // column tile, reduction length
  PS ps;
  QS qs;
  const uint8_t* P = static_cast<const uint8_t*>(a.p);
  const uint8_t* Q = static_cast<const uint8_t*>(a.q);
  if constexpr (OP == kWgrad) {
    // tile of group e: rows are N, columns K; XCD x takes a run of tiles
    const int nrow = (a.N + BM - 1) / BM;
    const long tiles = long(a.E) * nrow * ncol, per = (tiles + 7) / 8;
    const long t = long(blockIdx.x & 7) * per + (blockIdx.x >> 3);
    if (long(blockIdx.x >> 3) >= per || t >= tiles) return;
    pl.e = int(t / (long(nrow) * ncol));
    const int in = int(t - long(pl.e) * nrow * ncol);
    ct = in / nrow;
    const int rt = in % nrow;
    pl.row0 = rt * BM;
    pl.rows = min(BM, a.N - pl.row0);
    const int2 r = group_rows(a.offsets, pl.e, a.E, a.R);
    const int ra = __builtin_amdgcn_readfirstlane(r.x);
    red = __builtin_amdgcn_readfirstlane(r.y) - ra;
    ps.init(P + (long(ra) * a.N + pl.row0) * 2, (long(red) * a.N - pl.row0) * 2, long(a.N) * 2, w, lane, nullptr, 0, 0);
    qs.init(Q + (long(ra) * a.K + ct * kBN) * 2, (long(red) * a.K - ct * kBN) * 2, long(a.K) * 2, w, lane, nullptr, 0,
            0);
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
    if (pl.e == a.E) red = 0;  // rows behind the last group: zeros
  }
  const int steps = (red + kStep - 1) / kStep;

  typename Acc<TY>::type acc[MF][NF];
#pragma unroll
  for (int i = 0; i < MF; ++i)
#pragma unroll
    for (int j = 0; j < NF; ++j) acc[i][j] = typename Acc<TY>::type{0, 0, 0, 0};

  int kleft = red * kEl;  // bytes of a C row from this step on
  auto issue = [&](uint8_t* sp, uint8_t* sq) __attribute__((always_inline)) {
    ps.issue(sp, w, kleft);
    qs.issue(sq, w, kleft);
    ps.advance();
    qs.advance();
    kleft -= 128;
  };
  auto multiply = [&](const uint8_t* sp, const uint8_t* sq) __attribute__((always_inline)) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      v4i pf[MF], qf[NF];
#pragma unroll
      for (int j = 0; j < NF; ++j) qf[j] = read_frag<QT, kBN>(sq, wn * NF + j, kk, lane);
#pragma unroll
      for (int i = 0; i < MF; ++i) pf[i] = read_frag<PT, BM>(sp, wm * MF + i, kk, lane);
#pragma unroll
      for (int i = 0; i < MF; ++i)
#pragma unroll
        for (int j = 0; j < NF; ++j) acc[i][j] = mma<TY>(qf[j], pf[i], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };

  // a stage's barrier: its loads have arrived, the other stage is no longer read
  if (steps > 0) issue(p0, q0);
  int s = 0;
  for (; s + 1 < steps; s += 2) {
    stage_barrier();
    issue(p1, q1);
    multiply(p0, q0);
    stage_barrier();
    if (s + 2 < steps) issue(p0, q0);
    multiply(p1, q1);
  }
  if (s < steps) {
    stage_barrier();
    multiply(p0, q0);
  }

  // lane l holds column 4 (l / 16) + 0..3 and row l % 16 of each fragment
  const int m = lane & 15, g = lane >> 4;
  const long out_row0 = OP == kWgrad ? long(pl.e) * a.N + pl.row0 : long(pl.row0);
#pragma unroll
  for (int i = 0; i < MF; ++i) {
    const int r = wm * (BM / 2) + i * 16 + m;
    if (r >= pl.rows) continue;
    float sr = 0.0f;
    if constexpr (TY == kInt8) {
      if (pl.e < a.E) {
        const int t = a.row_token ? a.row_token[pl.row0 + r] : pl.row0 + r;
        if (!a.row_token || (t >= 0 && t < a.T)) sr = a.ps[t];
      }
    }
#pragma unroll
    for (int j = 0; j < NF; ++j) {
      const int c = ct * kBN + wn * 64 + j * 16 + 4 * g;
      if (c >= cols) continue;
      v4f v;
      if constexpr (TY == kInt8) {
        v = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        if (pl.e < a.E) {
          const v4f sc = *reinterpret_cast<const v4f*>(a.qs + long(pl.e) * a.N + c);
          v = __builtin_convertvector(acc[i][j], v4f) * sr * sc;
        }
      } else {
        v = acc[i][j];
      }
      store4(a.out, (out_row0 + r) * cols + c, v, a.out_ty);
    }
  }
}

int row_tile(int op, const MmArgs& a) {
  if (op == kWgrad) return 256;
  const long groups = a.E < a.R ? a.E : (a.R > 0 ? a.R : 1);
  const double avg = double(a.R) / double(groups);
  return avg >= 384 ? 256 : avg >= 96 ? 128 : 64;
}

}  // namespace

long mm_grid(int op, const MmArgs& a) {
  const int BM = row_tile(op, a);
  const long cols = op == kFwd ? a.N : a.K, ncol = (cols + kBN - 1) / kBN;
  long rows;
  if (op == kWgrad) {
    rows = long(a.E) * ((a.N + BM - 1) / BM);
  } else {
    // sum over non-empty groups (and the tail) of ceil(n / BM)
    const long G = (a.E < a.R ? a.E : a.R) + (a.clear_tail ? 1 : 0);
    const long most = (long(a.R) + G * (BM - 1)) / BM;
    rows = most < a.R ? most : a.R;
  }
  return (rows * ncol + 7) / 8 * 8;
}

template <int OP, int TY>
static hipError_t launch_bm(const MmArgs& a, hipStream_t st) {
  const unsigned grid = unsigned(mm_grid(OP, a));
  if constexpr (OP == kWgrad) {
    hipLaunchKernelGGL((k_mm<OP, TY, 256>), dim3(grid), dim3(kThreads), 0, st, a);
  } else {
    const int BM = row_tile(OP, a);
    if (BM == 256) hipLaunchKernelGGL((k_mm<OP, TY, 256>), dim3(grid), dim3(kThreads), 0, st, a);
    else if (BM == 128) hipLaunchKernelGGL((k_mm<OP, TY, 128>), dim3(grid), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_mm<OP, TY, 64>), dim3(grid), dim3(kThreads), 0, st, a);
  }
  return hipGetLastError();
}

hipError_t launch_mm(int op, const MmArgs& a, hipStream_t st) {
  if (mm_grid(op, a) == 0) return hipSuccess;
  if (a.ty == kInt8) return launch_bm<kFwd, kInt8>(a, st);
  if (a.ty == kBf16)
    return op == kFwd ? launch_bm<kFwd, kBf16>(a, st)
                      : op == kDgrad ? launch_bm<kDgrad, kBf16>(a, st) : launch_bm<kWgrad, kBf16>(a, st);
  return op == kFwd ? launch_bm<kFwd, kFp16>(a, st)
                    : op == kDgrad ? launch_bm<kDgrad, kFp16>(a, st) : launch_bm<kWgrad, kFp16>(a, st);
}

}  // namespace moe
