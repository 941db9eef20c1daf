// moe_few.hip -- the whole expert layer for up to 64 tokens on 16-bit row-major
// weights, in two launches:
//   h[t][j] = silu(W1g x[t]) * (W1u x[t])                     (k_up)
//   out[t]  = sum over j of weight[t][j] W2 h[t][j]           (k_down)
// with the matrices of expert id[t][j].
//
// Bound by the touched experts' weights, which are read once: lanes load matrix
// fragments straight into registers, several steps ahead, and nothing is shared
// between waves but their sums.  h stays exact enough for fp32 results: it is
// kept as the sum of two 16-bit values, and the second product takes both (the
// matrix units wait for memory here, so the second half costs nothing).
#include "moe_few.h"

#include "moe_mm_tile.h"
#include "moe_quant_i8.h"

namespace moe {
namespace {

constexpr int kRows = kFewTokens;  // rows of a tile: one tile per expert as long as no token names it twice
constexpr int kStep = 64;          // values of K per step: 128 bytes of a row

template <int TY>
__device__ __forceinline__ v4f mma16(const v4i& a, const v4i& b, const v4f& c) {
  if constexpr (TY == kBf16)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8v, a), __builtin_bit_cast(bf8v, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(h8v, a), __builtin_bit_cast(h8v, b), c, 0, 0, 0);
}

__device__ __forceinline__ v4i load16(const uint16_t* p) { return *reinterpret_cast<const v4i*>(p); }

// The fragments of one step: COLS operands of 16 weight rows, ROWS of 16 rows of
// the other operand, each in two halves of 32 values.
template <int COLS, int ROWS>
struct Step {
  v4i w[COLS][2], p[ROWS][2];
};

// acc[i][j] += over the steps [a, b) of K.  Lane l has row l % 16 of each fragment:
// w[i] and p[j] point to its row's value 8 (l / 16) of step 0; a step's second half lies
// 32 values on.  D steps are in flight.
template <int TY, int COLS, int ROWS, int D>
__device__ __forceinline__ void sum_steps(v4f (&acc)[COLS][ROWS], const uint16_t* const (&w)[COLS],
                                          const uint16_t* const (&p)[ROWS], int a, int b, int K) {
  typedef Step<COLS, ROWS> S;
  const int g = (threadIdx.x & 63) >> 4;
  const int full = K / kStep, n = min(b, full) - a;  // whole steps
  auto load = [&](S& s, int at) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < COLS; ++i) s.w[i][h] = load16(w[i] + long(at) * kStep + 32 * h);
#pragma unroll
      for (int j = 0; j < ROWS; ++j) s.p[j][h] = load16(p[j] + long(at) * kStep + 32 * h);
    }
  };
  auto use = [&](const S& s) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < COLS; ++i)
#pragma unroll
        for (int j = 0; j < ROWS; ++j) acc[i][j] = mma16<TY>(s.w[i][h], s.p[j][h], acc[i][j]);
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
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = full * kStep + 32 * h + 8 * g < K;
#pragma unroll
      for (int i = 0; i < COLS; ++i) s.w[i][h] = in ? load16(w[i] + long(full) * kStep + 32 * h) : v4i{0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < ROWS; ++j) s.p[j][h] = in ? load16(p[j] + long(full) * kStep + 32 * h) : v4i{0, 0, 0, 0};
    }
    use(s);
  }
}

// ------------------------------------------------------------------ first product
constexpr int kUpWaves = 4;
constexpr int kMaxExperts = 1024;

// 16 columns of h for one row tile: their gate and up rows of W1, K split over the
// waves, whose sums meet in LDS.
template <int TY, int NT, int D>
__device__ __forceinline__ void up_tile(const FewArgs& a, int e, int rows, int i0, const int* list, v4f* part) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, m = lane & 15, g = lane >> 4;
  const int col = min(i0 + m, a.I - 1);  // (columns behind the last are not stored)
  const uint16_t* w1 = static_cast<const uint16_t*>(a.w1) + long(e) * 2 * a.I * a.H + 8 * g;
  const uint16_t* const pw[2] = {w1 + long(col) * a.H, w1 + (long(a.I) + col) * a.H};
  const uint16_t* px[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = t * 16 + m;  // (rows behind the last take the first one's values, and are not stored)
    px[t] = static_cast<const uint16_t*>(a.x) + long(list[r < rows ? r : 0] / a.k) * a.H + 8 * g;
  }
  v4f acc[2][NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) acc[0][t] = acc[1][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  const int steps = (a.H + kStep - 1) / kStep;
  sum_steps<TY, 2, NT, D>(acc, pw, px, w * steps / kUpWaves, (w + 1) * steps / kUpWaves, a.H);
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int t = 0; t < NT; ++t) part[((w * 2 + c) * NT + t) * 64 + lane] = acc[c][t];
  __syncthreads();
  if (w < NT) {  // fragment w: lane l holds columns 4 (l / 16) + 0..3 of row l % 16
    v4f s[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      s[c] = part[(c * NT + w) * 64 + lane];
#pragma unroll
      for (int u = 1; u < kUpWaves; ++u) s[c] += part[((u * 2 + c) * NT + w) * 64 + lane];
    }
    const int r = w * 16 + m, c = i0 + 4 * g;
    if (r < rows && c < a.I) {
      v4f hi, lo;
      uint2 top;
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[j] = swiglu(s[0][j], s[1][j]);
      top = round4(hi, TY);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bits = (j < 2 ? top.x : top.y) >> (16 * (j & 1)) & 0xFFFFu;
        const float back = TY == kBf16 ? bf16_to_f32(bits) : float(__builtin_bit_cast(_Float16, uint16_t(bits)));
        lo[j] = fabsf(back) < __builtin_inff() ? hi[j] - back : 0.0f;  // (past the type's range: infinity)
      }
      const long at = long(list[r]) * a.I + c;
      *reinterpret_cast<uint2*>(a.hi + at) = top;
      *reinterpret_cast<uint2*>(a.lo + at) = round4(lo, TY);
    }
  }
}

// A workgroup finds its row tile from the routing result itself: experts' counts,
// then the tile's expert, then its slots in their order.  The workgroups of the
// first columns write that down for the second launch.
template <int TY>
__global__ __launch_bounds__(kUpWaves * 64) void k_up(FewArgs a, int ncol) {
  __shared__ int hist[kMaxExperts];
  __shared__ int list[kRows];
  __shared__ v4f part[kUpWaves * 2 * (kRows / 16) * 64];
  const int lane = threadIdx.x & 63, n = a.T * a.k;
  const int want = int(blockIdx.x) / ncol, ct = int(blockIdx.x) - want * ncol;
  for (int e = threadIdx.x; e < a.E; e += kUpWaves * 64) hist[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kUpWaves * 64) {
    const int id = a.ids[i];
    if (id >= 0 && id < a.E) atomicAdd(&hist[id], 1);
  }
  __syncthreads();
  // tile `want`: expert e and the rows of its tiles before (every wave by itself)
  int before = 0, e = -1, skip = 0, rows = 0;
  for (int e0 = 0; e0 < a.E; e0 += 64) {
    const int c = e0 + lane < a.E ? hist[e0 + lane] : 0;
    int tiles = (c + kRows - 1) / kRows, incl = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int v = __shfl_up(incl, d, 64);
      if (lane >= d) incl += v;
    }
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
      const bool mine = i0 + lane < n && a.ids[i0 + lane] == e;
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
  if (rows <= 16) up_tile<TY, 1, 4>(a, e, rows, ct * 16, list, part);
  else if (rows <= 32) up_tile<TY, 2, 3>(a, e, rows, ct * 16, list, part);
  else up_tile<TY, 4, 2>(a, e, rows, ct * 16, list, part);
}

// ------------------------------------------------------------------ second product
constexpr int kDownWaves = 8;

// Steps [s0, s1) of row tile v for 16 columns of out, added to the wave's own sums
// by token.
template <int TY, int NT, int D>
__device__ __forceinline__ void down_tile(const FewArgs& a, int v, int e, int rows, int n0, int s0, int s1,
                                          float (*sums)[16]) {
  const int lane = threadIdx.x & 63, m = lane & 15, g = lane >> 4;
  const int col = min(n0 + m, a.H - 1);
  const uint16_t* const pw[1] = {static_cast<const uint16_t*>(a.w2) + (long(e) * a.H + col) * a.I + 8 * g};
  const uint16_t* ph[2 * NT];
  int slot[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int r = t * 16 + m;
    slot[t] = a.slots[v * kRows + (r < rows ? r : 0)];
    ph[t] = a.hi + long(slot[t]) * a.I + 8 * g;
    ph[NT + t] = a.lo + long(slot[t]) * a.I + 8 * g;
  }
  v4f acc[1][2 * NT];
#pragma unroll
  for (int t = 0; t < 2 * NT; ++t) acc[0][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  sum_steps<TY, 1, 2 * NT, D>(acc, pw, ph, s0, s1, a.I);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    if (t * 16 + m < rows) {
      const float weight = a.weights[slot[t]];
      float* to = sums[slot[t] / a.k] + 4 * g;
#pragma unroll
      for (int j = 0; j < 4; ++j)  // (two rows of a tile may be one token's)
        __hip_atomic_fetch_add(to + j, weight * (acc[0][t][j] + acc[0][NT + t][j]), __ATOMIC_RELAXED,
                               __HIP_MEMORY_SCOPE_WORKGROUP);
    }
  }
}

// 16 columns of out: all steps of all row tiles in one row, an eighth of them to
// each wave.
template <int TY>
__global__ __launch_bounds__(kDownWaves * 64) void k_down(FewArgs a) {
  __shared__ float sums[kDownWaves][kFewTokens][16];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), n0 = int(blockIdx.x) * 16;
  for (int i = threadIdx.x & 63; i < a.T * 16; i += 64) sums[w][i / 16][i % 16] = 0.0f;
  const int each = (a.I + kStep - 1) / kStep;
  const long total = long(*a.count) * each;
  long at = total * w / kDownWaves;
  const long end = total * (w + 1) / kDownWaves;
  while (at < end) {
    const int v = int(at / each), s0 = int(at - long(v) * each), s1 = int(min(long(each), s0 + end - at));
    const int2 tile = a.tiles[v];
    if (tile.y <= 16) down_tile<TY, 1, 4>(a, v, tile.x, tile.y, n0, s0, s1, sums[w]);
    else if (tile.y <= 32) down_tile<TY, 2, 2>(a, v, tile.x, tile.y, n0, s0, s1, sums[w]);
    else down_tile<TY, 4, 1>(a, v, tile.x, tile.y, n0, s0, s1, sums[w]);
    at += s1 - s0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.T * 4; i += kDownWaves * 64) {
    const int t = i / 4, c = i % 4 * 4;
    v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int u = 0; u < kDownWaves; ++u) s += *reinterpret_cast<const v4f*>(&sums[u][t][c]);
    if (n0 + c < a.H) store4(a.out, long(t) * a.H + n0 + c, s, TY);
  }
}

// Row tiles at most: each expert has one more than it fills.
long most_tiles(int T, int E, int k) {
  const long n = long(T) * k, most = (E < n ? E : n) + n / kRows;
  return most < n ? most : n;
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

template <int TY>
hipError_t launch_ty(const FewArgs& a, hipStream_t st) {
  const int ncol = (a.I + 15) / 16;
  hipLaunchKernelGGL((k_up<TY>), dim3(unsigned(most_tiles(a.T, a.E, a.k) * ncol)), dim3(kUpWaves * 64), 0, st, a, ncol);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_down<TY>), dim3(unsigned((a.H + 15) / 16)), dim3(kDownWaves * 64), 0, st, a);
  return hipGetLastError();
}

}  // namespace

size_t few_bytes(int T, int I, int E, int k) {
  const size_t tiles = size_t(most_tiles(T, E, k));
  return 256 + up256(tiles * sizeof(int2)) + up256(tiles * kRows * 4) + 2 * up256(size_t(T) * k * I * 2);
}

void few_carve(FewArgs& a, void* ws) {
  const size_t tiles = size_t(most_tiles(a.T, a.E, a.k));
  uint8_t* p = static_cast<uint8_t*>(ws);
  a.count = reinterpret_cast<int32_t*>(p);
  p += 256;
  a.tiles = reinterpret_cast<int2*>(p);
  p += up256(tiles * sizeof(int2));
  a.slots = reinterpret_cast<int32_t*>(p);
  p += up256(tiles * kRows * 4);
  a.hi = reinterpret_cast<uint16_t*>(p);
  p += up256(size_t(a.T) * a.k * a.I * 2);
  a.lo = reinterpret_cast<uint16_t*>(p);
}

hipError_t launch_few(const FewArgs& a, hipStream_t st) {
  return a.ty == kBf16 ? launch_ty<kBf16>(a, st) : launch_ty<kFp16>(a, st);
}

}  // namespace moe
