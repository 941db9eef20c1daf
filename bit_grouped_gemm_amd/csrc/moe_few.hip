// moe_few.hip -- the whole expert layer for up to 64 tokens on 16-bit row-major
// weights, in two launches, or three:
//   h[t][j] = silu(W1g x[t]) * (W1u x[t])                     (k_up)
//   out[t]  = sum over j of weight[t][j] W2 h[t][j]           (k_down, k_down_join)
// with the matrices of expert id[t][j].
//
// Bound by the touched experts' weights, which are read once for each tile of rows (as a
// rule an expert has one): lanes load matrix operands straight into registers, several
// steps ahead, and nothing is shared between waves but their sums.  h is kept as the sum of
// two 16-bit values, and the second product takes both (the matrix units wait for memory
// here, so the second half costs nothing): 2^-17 of it is lost in bf16, 2^-21 in fp16, where
// the lower value ends at 2^-24, so that an h below some 2^-14 is an fp16 value, and one past
// 65504 is infinite.
//
// A 16 x 16 x 32 product takes 16 rows of 64 bytes, which is half of each line: the other
// half then waits in the L1 for the next load, among those of a dozen waves, and is
// often gone (four steps ahead were slower than two).  So a load has eight rows of 128
// bytes, and the product's 16 rows are their two halves: row 2 r + s is half s of row r.
// The other operand is laid out alike, and of the 16 x 16 sums those of equal
// halves are the ones that are meant; the two of a row are added up at the end.
//
// One bf16 token, 8 of 64 experts, H=4096, I=1408: k_up 31 us, 6.0 TB/s of weights, k_down 17,
// 5.4 (half lines: 40 and 21; a stream of plain reads reaches 6.9 TB/s).  8 tokens that name each
// expert once: 212, 7.0 TB/s, and 115, 6.4; 61 tokens, popular experts named more often: 231 to 280 from
// process to process, 6.4 to 5.3, and 122 to 154 + 5: the rows of x and h take their share of what reaches a CU.
// Rows that are no whole lines (H or I no multiple of 64) cost half as much again and more: 8 tokens, H=4096,
// I=1408, 45 experts 162 and 83 us, 6.4 and 6.3 TB/s; H=4104, I=1416, 39 experts 226 and 110, 4.0 and 4.1.
#include <cmath>

#include "moe_few.h"

#include "moe_mm_tile.h"
#include "moe_quant_i8.h"

namespace moe {
namespace {

// Rows of a tile, for T tokens: the fewest that hold what an expert gets as a rule (a
// token names it once), as the sums of more would cost every wave the registers that keep
// its loads in flight.  From 33 tokens on an expert that most of them name has two
// tiles, and its weights are read twice.
constexpr int tile_rows(int T) { return T <= 8 ? 8 : T <= 16 ? 16 : 32; }
constexpr int kStep = 64;          // values of K per step: 128 bytes of a row

template <int TY>
__device__ __forceinline__ v4f mma16(const v4i& a, const v4i& b, const v4f& c) {
  if constexpr (TY == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, a), __builtin_bit_cast(h8v, b), c, 0, 0, 0);
}

__device__ __forceinline__ v4i load16(const uint16_t* p) { return *reinterpret_cast<const v4i*>(p); }
// the same of weights: read once, so not kept in the caches
__device__ __forceinline__ v4i stream16(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p));
}

// This lane's row of a group of eight, and the first value of its 16 bytes of a step.
__device__ __forceinline__ int row_of() { return int(threadIdx.x & 15) >> 1; }
__device__ __forceinline__ int chunk_of() { return 8 * (4 * int(threadIdx.x & 1) + (int(threadIdx.x & 63) >> 4)); }

// One step of NW groups of eight weight rows and NP groups of eight rows of the other operand.
template <int NW, int NP>
struct Step {
  v4i w[NW], p[NP];
};

// acc[i][j % NA] += over the steps [a, b) of K.  Lane l has row (l % 16) / 2 of each group, and of
// its step the 16 bytes 4 (l % 2) + l / 16; w[i] and p[j] point to them in step 0.  D steps
// are in flight.
template <int TY, int NW, int NP, int D, int NA>
__device__ __forceinline__ void sum_steps(v4f (&acc)[NW][NA], const uint16_t* const (&w)[NW],
                                          const uint16_t* const (&p)[NP], int a, int b, int K) {
  typedef Step<NW, NP> S;
  const int full = K / kStep, n = min(b, full) - a;  // whole steps
  auto load = [&](S& s, int at) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NW; ++i) s.w[i] = stream16(w[i] + long(at) * kStep);
#pragma unroll
    for (int j = 0; j < NP; ++j) s.p[j] = load16(p[j] + long(at) * kStep);
  };
  auto use = [&](const S& s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int j = 0; j < NP; ++j) acc[i][j % NA] = mma16<TY>(s.w[i], s.p[j], acc[i][j % NA]);
  };
  if (n > 0) {
    S s[D];
#pragma unroll
    for (int d = 0; d < D; ++d) load(s[d], a + min(d, n - 1));
    int k = 0;
    for (; k + D <= n; k += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        use(s[d]);
        load(s[d], a + min(k + d + D, n - 1));  // (the last ones again where there are no more)
      }
    }
#pragma unroll
    for (int d = 0; d < D; ++d)
      if (k + d < n) use(s[d]);
  }
  if (b > full && b > a && K % kStep) {  // the rest of K: zeros behind it
    S s;
    const bool in = full * kStep + chunk_of() < K;
#pragma unroll
    for (int i = 0; i < NW; ++i) s.w[i] = in ? stream16(w[i] + long(full) * kStep) : v4i{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < NP; ++j) s.p[j] = in ? load16(p[j] + long(full) * kStep) : v4i{0, 0, 0, 0};
    use(s);
  }
}

// The sums of a group of weight rows with a group of the others: lane l has weight
// rows 2 (l / 16) and 2 (l / 16) + 1 of the other's row (l % 16) / 2.
__device__ __forceinline__ float2 both_halves(const v4f& acc) {
  const bool s = threadIdx.x & 1;
  const float x = s ? acc[1] : acc[0], y = s ? acc[3] : acc[2];
  return make_float2(x + dpp_f32<0xB1>(x), y + dpp_f32<0xB1>(y));  // (lane xor 1)
}

// ------------------------------------------------------------------ first product
// (Steps in flight for up to 8, 16 and 32 rows, us for 61 tokens as listed above, and for 64 with 16 rows for each
// of 32 experts: 3, 2, 2 277 and 134; 3, 3, 1 276 and 131; 4, 3, 2 287 and 131; 2, 2, 1 285 and
// 132; 2, 1, 1 306 and 150.  32 columns a workgroup, which halves the reads of x: 290 and 145, as its
// registers leave one wave per SIMD.  One token, steps: 2 31.2, 3 30.8, 6 30.6, 8 35.)
constexpr int kUpWaves = 4, kUpCols = 16;
constexpr int kMaxExperts = 1024, kMaxTopk = 32;

// 16 columns of h for one row tile: their gate and up rows of W1, K split over the
// waves, whose sums meet in LDS.
template <int TY, int NP, int D>
__device__ __forceinline__ void up_tile(const FewArgs& a, int e, int rows, int i0, const int* list, float2* part) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const uint16_t* w1 = static_cast<const uint16_t*>(a.w1) + long(e) * 2 * a.I * a.H + chunk_of();
  constexpr int NW = kUpCols / 4;  // groups of eight rows: the gate rows', then the up rows'
  const uint16_t* pw[NW];
#pragma unroll
  for (int i = 0; i < NW / 2; ++i) {
    const int col = min(i0 + i * 8 + row_of(), a.I - 1);  // (columns behind the last are not stored)
    pw[i] = w1 + long(col) * a.H;
    pw[NW / 2 + i] = w1 + (long(a.I) + col) * a.H;
  }
  const uint16_t* px[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int r = j * 8 + row_of();  // (rows behind the last take the first one's values, and are not stored)
    px[j] = static_cast<const uint16_t*>(a.x) + long(list[r < rows ? r : 0] / a.k) * a.H + chunk_of();
  }
  v4f acc[NW][NP];
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (a.H + kStep - 1) / kStep;
  sum_steps<TY, NW, NP, D>(acc, pw, px, w * steps / kUpWaves, (w + 1) * steps / kUpWaves, a.H);
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) part[((w * NW + i) * NP + j) * 64 + lane] = both_halves(acc[i][j]);
  __syncthreads();
  for (int f = w; f < NW / 2 * NP; f += kUpWaves) {  // eight columns of eight rows
    const int i = f / NP, j = f % NP;
    float2 gate = {0.0f, 0.0f}, up = {0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kUpWaves; ++u) {
      const float2 g = part[((u * NW + i) * NP + j) * 64 + lane];
      const float2 v = part[((u * NW + NW / 2 + i) * NP + j) * 64 + lane];
      gate.x += g.x;
      gate.y += g.y;
      up.x += v.x;
      up.y += v.y;
    }
    const int r = j * 8 + row_of(), c = i0 + i * 8 + 2 * (lane >> 4);
    if (r >= rows || c >= a.I || (lane & 1)) continue;
    const v4f h = {swiglu(gate.x, up.x), swiglu(gate.y, up.y), 0.0f, 0.0f};
    const uint32_t hi = round4(h, TY).x;
    v4f lo = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const uint32_t bits = hi >> (16 * u) & 0xFFFFu;
      const float back = TY == kBf16 ? bf16_to_f32(bits) : float(__builtin_bit_cast(_Float16, uint16_t(bits)));
      lo[u] = fabsf(back) < __builtin_inff() ? h[u] - back : 0.0f;  // (past the type's range: infinity)
    }
    const long at = long(list[r]) * a.I + c;
    *reinterpret_cast<uint32_t*>(a.hi + at) = hi;
    *reinterpret_cast<uint32_t*>(a.lo + at) = round4(lo, TY).x;
  }
}

// A workgroup finds its row tile from the routing result itself: experts' counts,
// then the tile's expert, then its slots in their order.  The workgroups of the
// first columns write that down for the second launch.
template <int TY, int MAXP>
__global__ __launch_bounds__(kUpWaves * 64, 3) void k_up(FewArgs a, int ncol) {
  constexpr int kRows = 8 * MAXP;
  __shared__ int hist[kMaxExperts];
  __shared__ int list[kRows];
  __shared__ int16_t named[kFewTokens * kMaxTopk];  // a slot's expert, or -1
  __shared__ float2 part[kUpWaves * (kUpCols / 4) * MAXP * 64];
  const int lane = threadIdx.x & 63, n = a.T * a.k;
  const int want = int(blockIdx.x) / ncol, ct = int(blockIdx.x) - want * ncol;
  for (int e = threadIdx.x; e < a.E; e += kUpWaves * 64) hist[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kUpWaves * 64) {
    const int id = a.ids[i];
    const bool live = id >= 0 && id < a.E;
    named[i] = int16_t(live ? id : -1);
    if (live) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  // tile `want`: expert e and the rows of its tiles before (every wave by itself)
  int before = 0, e = -1, skip = 0, rows = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int c = e0 + lane < a.E ? hist[e0 + lane] : 0;
    const int tiles = (c + kRows - 1) / kRows, incl = wave_scan_sat(tiles);
    const uint64_t past = __ballot(before + incl > want);
    if (past && e < 0) {
      const int l = __ffsll((unsigned long long)past) - 1;
      const int first = before + __builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(tiles, l);
      e = e0 + l;
      skip = (want - first) * kRows;
      rows = min(kRows, __builtin_amdgcn_readlane(c, l) - skip);
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  const bool notes = ct == 0 && threadIdx.x < 64;
  if (notes && want == 0 && lane == 0) *a.count = before;
  if (e < 0) return;
  if (threadIdx.x < 64) {
    for (int i0 = 0, seen = 0; i0 < n; i0 += 64) {
      const bool mine = i0 + lane < n && named[i0 + lane] == e;
      const uint64_t all = __ballot(mine);
      const int at = seen + __popcll(all & ((1ull << lane) - 1)) - skip;
      if (mine && at >= 0 && at < rows) {
        list[at] = i0 + lane;
        if (notes) a.slots[want * kRows + at] = i0 + lane;
      }
      seen += __popcll(all);
    }
    if (notes && lane == 0) a.tiles[want] = make_int2(e, rows);
  }
  __syncthreads();
  const int i0 = ct * kUpCols;
  if (MAXP == 1 || rows <= 8) up_tile<TY, 1, 3>(a, e, rows, i0, list, part);
  else if (MAXP == 2 || rows <= 16) up_tile<TY, MAXP < 2 ? MAXP : 2, 2>(a, e, rows, i0, list, part);
  else up_tile<TY, MAXP, 2>(a, e, rows, i0, list, part);
}

// ------------------------------------------------------------------ second product
// (Steps in flight, us for one token: 4 16.9, 6 16.8, 8 16.8, 16 waves with 4 17.1; for 61, up to 8 rows
// and up to 16: 3 and 2 152, 3 and 3 148, 4 and 2 153, 5 and 4 151.)
constexpr int kDownWaves = 8;

// Steps [s0, s1) of a row tile for 8 NW columns of out, added to the wave's own sums
// by token.
template <int TY, int NW, int NP, int D>
__device__ __forceinline__ void down_tile(const FewArgs& a, const int* slots, int e, int rows, int n0, int s0, int s1,
                                          float (*sums)[8 * NW]) {
  const int lane = threadIdx.x & 63;
  const uint16_t* w2 = static_cast<const uint16_t*>(a.w2) + long(e) * a.H * a.I + chunk_of();
  const uint16_t* pw[NW];
#pragma unroll
  for (int i = 0; i < NW; ++i) pw[i] = w2 + long(min(n0 + i * 8 + row_of(), a.H - 1)) * a.I;
  const uint16_t* ph[2 * NP];
  int slot[NP];
  float weight[NP];
  const int first = __builtin_amdgcn_readfirstlane(slots[0]);  // (for the rows behind the last)
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    slot[j] = j * 8 + row_of() < rows ? slots[j] : first;
    weight[j] = a.weights[slot[j]];
    ph[j] = a.hi + long(slot[j]) * a.I + chunk_of();
    ph[NP + j] = a.lo + long(slot[j]) * a.I + chunk_of();
  }
  v4f acc[NW][NP];
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int j = 0; j < NP; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  sum_steps<TY, NW, 2 * NP, D>(acc, pw, ph, s0, s1, a.I);
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const bool mine = j * 8 + row_of() < rows && !(lane & 1);
    float* to = sums[slot[j] / a.k] + 2 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const float2 y = both_halves(acc[i][j]);
      if (mine) {  // (two rows of a tile may be one token's)
        __hip_atomic_fetch_add(to + i * 8, weight[j] * y.x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        __hip_atomic_fetch_add(to + i * 8 + 1, weight[j] * y.y, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      }
    }
  }
}

// 8 NW columns of out: all steps of all row tiles in one row.  The workgroups have equal shares of
// all columns' steps, and a workgroup's waves of its own.
// Columns that one workgroup has alone it writes, of others their sums so far.
template <int TY, int MAXP, int NW>
__global__ __launch_bounds__(kDownWaves * 64) void k_down(FewArgs a, int ncol) {
  constexpr int kCols = 8 * NW;
  __shared__ float sums[kDownWaves][kFewTokens][kCols];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int each = (a.I + kStep - 1) / kStep, count = *a.count;
  const long total = max(long(count) * each, 1L), end = total * ncol * (blockIdx.x + 1) / gridDim.x;
  struct Tile {
    int e, rows, slots[MAXP];  // this lane's rows' slots (anything behind the last row)
  };
  // (all its loads at once, and a tile ahead: 19 tokens 116 us, 119 with each when it is needed)
  auto tile_at = [&](int v) __attribute__((always_inline)) {
    Tile t;
    const int2 head = a.tiles[v];
    t.e = head.x;
    t.rows = head.y;
#pragma unroll
    for (int j = 0; j < MAXP; ++j) t.slots[j] = a.slots[(v * MAXP + j) * 8 + row_of()];
    return t;
  };
  int turn = 0;
  for (long u = total * ncol * blockIdx.x / gridDim.x; u < end; ++turn) {
    const int ct = int(u / total), n0 = ct * kCols;
    const int from = int(u - ct * total), upto = int(min(total, from + end - u));
    for (int i = lane; i < a.T * kCols; i += 64) sums[w][i / kCols][i % kCols] = 0.0f;
    int at = from + int(long(upto - from) * w / kDownWaves);
    const int last = count ? from + int(long(upto - from) * (w + 1) / kDownWaves) : at;
    Tile next = at < last ? tile_at(at / each) : Tile{};
    while (at < last) {
      const int v = at / each, s0 = at - v * each, s1 = min(each, s0 + last - at);
      const Tile now = next;
      at += s1 - s0;
      if (at < last) next = tile_at(v + 1);
      const int e = __builtin_amdgcn_readfirstlane(now.e), rows = __builtin_amdgcn_readfirstlane(now.rows);
      constexpr int D = NW == 2 ? 6 : 3;
      if (MAXP == 1 || rows <= 8) down_tile<TY, NW, 1, D>(a, now.slots, e, rows, n0, s0, s1, sums[w]);
      else if (MAXP == 2 || rows <= 16)
        down_tile<TY, NW, MAXP < 2 ? 1 : 2, D>(a, now.slots, e, rows, n0, s0, s1, sums[w]);
      else down_tile<TY, NW, MAXP, 2>(a, now.slots, e, rows, n0, s0, s1, sums[w]);
    }
    __syncthreads();
    const bool whole = from == 0 && upto == total;
    float* to = a.partial + (long(blockIdx.x) * 2 + (turn ? 1 : 0)) * a.T * kCols;
    for (int i = threadIdx.x; i < a.T * (kCols / 4); i += kDownWaves * 64) {
      const int t = i / (kCols / 4), c = i % (kCols / 4) * 4;
      v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < kDownWaves; ++x) s += *reinterpret_cast<const v4f*>(&sums[x][t][c]);
      if (!whole) *reinterpret_cast<v4f*>(to + t * kCols + c) = s;
      else if (n0 + c < a.H) store4(a.out, long(t) * a.H + n0 + c, s, TY);
    }
    __syncthreads();
    u += upto - from;
  }
}

// Columns that several workgroups have parts of: their sums, in the order of the workgroups.
template <int TY, int NW>
__global__ __launch_bounds__(256) void k_down_join(FewArgs a, int ncol, int blocks) {
  constexpr int kCols = 8 * NW;
  const int each = (a.I + kStep - 1) / kStep, ct = blockIdx.x;
  const long total = max(long(*a.count) * each, 1L), all = total * ncol;
  int b = int(long(ct) * blocks / ncol);  // the first one with steps of [ct total, (ct + 1) total)
  while (b > 0 && all * b / blocks > ct * total) --b;
  while (all * (b + 1) / blocks <= ct * total) ++b;
  if (all * b / blocks <= ct * total && all * (b + 1) / blocks >= (ct + 1) * total) return;  // has them alone
  for (int i = threadIdx.x; i < a.T * (kCols / 4); i += 256) {
    const int t = i / (kCols / 4), c = i % (kCols / 4) * 4;
    v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int v = b; v < blocks && all * v / blocks < (ct + 1) * total; ++v) {
      if (all * (v + 1) / blocks == all * v / blocks) continue;  // (without steps)
      const int turn = all * v / blocks >= ct * total ? 0 : 1;
      s += *reinterpret_cast<const v4f*>(a.partial + ((long(v) * 2 + turn) * a.T + t) * kCols + c);
    }
    if (ct * kCols + c < a.H) store4(a.out, long(t) * a.H + ct * kCols + c, s, TY);
  }
}

// Row tiles at most: each expert has one more than it fills.
long most_tiles(int T, int E, int k) {
  const long n = long(T) * k, most = (E < n ? E : n) + n / tile_rows(T);
  return most < n ? most : n;
}

// Columns and workgroups of the second product.  From 9 tokens on a workgroup has 32 columns, as it
// reads h for each 16 (32: 19 tokens, top-8 of 64, half of them here, 7168 x 2048, 119 us, 16: 145); one
// token's 16 fill more CUs.  Where the columns leave CUs idle, the workgroups are one per CU
// and share columns, if that saves more than the launch that adds up their sums: us, 8 tokens on all of 64 experts,
// 2048 x 1408: 91 whole, 58 + 5 shared; 61 tokens, 4096 x 1408: 221, 148 + 5; one token, 7168
// x 2048 (448 workgroups on 256 CUs): 46, 42 + 5.
struct DownShape {
  int cols, blocks;
  bool shared;
};
DownShape down_shape(int T, int H, int I, int E, int k) {
  const int cols = tile_rows(T) == 8 ? 16 : 32, tiles = (H + cols - 1) / cols;
  const double fill = tiles / (std::ceil(tiles / kCUs) * kCUs);  // of the CUs, over the rounds
  const double touched = E * (1.0 - std::exp(-double(T) * k / E)), whole = touched * H * I * 2 / 5.5e6;  // us
  const bool shared = tiles % int(kCUs) && fill < 0.85 && whole * (0.85 / fill - 1.0) > 6.0;
  return {cols, shared ? int(kCUs) : tiles, shared};
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

template <int TY, int MAXP>
hipError_t launch_rows(const FewArgs& a, hipStream_t st) {
  constexpr int NW = MAXP == 1 ? 2 : 4;
  const int up_tiles = (a.I + kUpCols - 1) / kUpCols;
  hipLaunchKernelGGL((k_up<TY, MAXP>), dim3(unsigned(most_tiles(a.T, a.E, a.k) * up_tiles)), dim3(kUpWaves * 64), 0, st,
                     a, up_tiles);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const DownShape s = down_shape(a.T, a.H, a.I, a.E, a.k);
  const int ncol = (a.H + 8 * NW - 1) / (8 * NW);
  hipLaunchKernelGGL((k_down<TY, MAXP, NW>), dim3(unsigned(s.blocks)), dim3(kDownWaves * 64), 0, st, a, ncol);
  e = hipGetLastError();
  if (e != hipSuccess || !s.shared) return e;
  hipLaunchKernelGGL((k_down_join<TY, NW>), dim3(unsigned(ncol)), dim3(256), 0, st, a, ncol, s.blocks);
  return hipGetLastError();
}

template <int TY>
hipError_t launch_ty(const FewArgs& a, hipStream_t st) {
  switch (tile_rows(a.T)) {
    case 8: return launch_rows<TY, 1>(a, st);
    case 16: return launch_rows<TY, 2>(a, st);
    default: return launch_rows<TY, 4>(a, st);
  }
}

}  // namespace

size_t few_bytes(int T, int H, int I, int E, int k) {
  const size_t tiles = size_t(most_tiles(T, E, k));
  const DownShape s = down_shape(T, H, I, E, k);
  return 256 + up256(tiles * sizeof(int2)) + up256(tiles * tile_rows(T) * 4) +
         2 * up256(size_t(T) * k * I * 2) + (s.shared ? size_t(s.blocks) * 2 * T * s.cols * 4 : 0);
}

void few_carve(FewArgs& a, void* ws) {
  const size_t tiles = size_t(most_tiles(a.T, a.E, a.k)), h = up256(size_t(a.T) * a.k * a.I * 2);
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.count = reinterpret_cast<int32_t*>(p);
  p += 256;
  a.tiles = reinterpret_cast<int2*>(p);
  p += up256(tiles * sizeof(int2));
  a.slots = reinterpret_cast<int32_t*>(p);
  p += up256(tiles * tile_rows(a.T) * 4);
  a.hi = reinterpret_cast<uint16_t*>(p);
  a.lo = reinterpret_cast<uint16_t*>(p + h);
  a.partial = reinterpret_cast<float*>(p + 2 * h);
}

hipError_t launch_few(const FewArgs& a, hipStream_t st) {
  return a.ty == kBf16 ? launch_ty<kBf16>(a, st) : launch_ty<kFp16>(a, st);
}

}  // namespace moe
