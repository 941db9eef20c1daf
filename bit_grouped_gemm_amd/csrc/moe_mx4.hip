// moe_mx4.hip -- MXFP4 on row-major operands: the quantiser of 16-bit rows and
// the product over ragged groups of rows.
//
//   y[r][n] = sum over blocks b of 32 of 2^(pe[r][b] - 127) 2^(qe[n][b] - 127)
//             sum_{k in b} p[r][k] q[n][k],   p and q e2m1 codes, sums in fp32
//
// The scaled matrix instruction takes the codes and the scales as they are.  It
// sums over K in any order as long as both operands agree, so a lane takes
// neighbouring blocks of its row in successive instructions: their scales are then
// neighbouring bytes, one read of which serves all of them.
#include <cmath>
#include <type_traits>

#include "moe_mm_tile.h"
#include "moe_mx4.h"
#include "moe_quant_mx4.h"

namespace moe {
namespace {

// ------------------------------------------------------------------ quantiser
// Eight values a lane, four lanes a block.  Bound by HBM: 2 (SwiGLU: 4) bytes in
// and 17/32 out per value.
constexpr int kQuantUnroll = 4;

template <int TY, bool GLU>
__global__ __launch_bounds__(256) void k_quant_mx4(const uint16_t* __restrict__ x, long chunks, int K,
                                                   uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  const int row_chunks = K / 8;
  const long step = long(gridDim.x) * 256 * kQuantUnroll;
  for (long at = long(blockIdx.x) * 256 * kQuantUnroll + threadIdx.x; at - threadIdx.x < chunks; at += step) {
    quant_raw8 v[kQuantUnroll], up[kQuantUnroll];
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
      const long i = at + u * 256;
      v[u] = up[u] = quant_raw8{0, 0, 0, 0};
      if (i < chunks) {
        const uint16_t* from = x + i * 8;
        if constexpr (GLU) from += i / row_chunks * K;
        v[u] = *reinterpret_cast<const quant_raw8*>(from);
        if constexpr (GLU) up[u] = *reinterpret_cast<const quant_raw8*>(from + K);
      }
    }
#pragma unroll
    for (int u = 0; u < kQuantUnroll; ++u) {
      const long i = at + u * 256;
      const f8v f = quant_value8<TY, GLU>(v[u], up[u]);
      const uint32_t scale = mx4_scale(group_top_dpp(quant_top8(f), 4));
      const uint32_t q = mx4_codes8(f, scale);
      if (i < chunks) {
        *reinterpret_cast<uint32_t*>(codes + i * 4) = q;
        if ((i & 3) == 0) scales[i >> 2] = uint8_t(scale);
      }
    }
  }
}

// ------------------------------------------------------------------ products
// A K step is 128 bytes of a row, 256 values, 8 blocks; scales come for four
// steps at a time, 32 bytes of a row.
constexpr int kGroupSteps = 4;

// 16 scale bytes of a row, wherever they lie; those from `left` on are zeros (their
// codes are).
__device__ __forceinline__ v4i load_scales16(const uint8_t* p, int left) {
  v4i v = {0, 0, 0, 0};
  if (left >= 16) {
    __builtin_memcpy(&v, p, 16);
  } else {
#pragma unroll
    for (int i = 0; i < 15; ++i)
      if (i < left) v[i >> 2] |= int(uint32_t(p[i]) << (8 * (i & 3)));
  }
  return v;
}

__device__ __forceinline__ v8i operand(const v4i& v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

// Whether row t of p, named by row_token, is one.
__device__ __forceinline__ int token_of(const Mx4Args& a, int row) {
  if (!a.row_token) return row;
  const int t = a.row_token[row];
  return t >= 0 && t < a.T ? t : -1;
}

// Where there are too few tiles for the chip: a workgroup makes 16 NC columns by
// 16 NT rows; each of its four waves takes a quarter of the K steps through a
// ring of S stages of its own, and their sums are added up, in the order of the
// waves, through LDS.
constexpr int kFewWaves = 4;

template <int NC, int NT, int S>
__global__ __launch_bounds__(kFewWaves * 64) void k_mx4_few(Mx4Args a) {
  constexpr int L = 2 * (NC + NT);            // loads of a wave per step
  constexpr int kStage = L * 1024;            // bytes of a wave's stage
  constexpr int kSets = (NC + NT + 1) / 2;    // loads of a wave per four steps of scales: 32 rows each
  constexpr int kScales = kSets * 1024;
  // one array per stage: the compiler's alias analysis then keeps a stage's
  // reads free of waits for the other stage's loads
  __shared__ __align__(1024) uint8_t st0[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st1[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st2[S == 4 ? kFewWaves * kStage : 16];
  __shared__ __align__(1024) uint8_t st3[S == 4 ? kFewWaves * kStage : 16];
  __shared__ __align__(1024) uint8_t scales[kFewWaves * kScales];
  static_assert((S == 2 || S == 4) && (S - 1) * L < 64, "ring");
  static_assert(NC * NT * 1024 <= kStage, "a wave's sums fit a stage");
  static_assert(kGroupSteps % S == 0, "the loop takes whole groups");
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int ncol = (a.N + 16 * NC - 1) / (16 * NC);
  Place pl;
  int ct;
  if (!find_tile(a, 16 * NT, ncol, blockIdx.x, pl, ct)) return;
  const int ld = a.K / 2, nb = a.K / 32;  // bytes of codes and of scales per row of both operands
  const int n0 = ct * 16 * NC;
  const int steps = pl.e >= a.E ? 0 : (ld + 127) / 128;
  const int each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = w * each, mine = max(0, min(steps - s0, each));

  const uint8_t* wq = static_cast<const uint8_t*>(a.q) + (long(pl.e) * a.N + n0) * ld;
  const int wrows = min(16 * NC, a.N - n0);
  const uint32_t wspan = uint32_t(wrows) * uint32_t(ld);
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
    if (a.row_token) t = r < pl.rows ? token_of(a, pl.row0 + r) : -1;
    op[i] = r < pl.rows && t >= 0 ? uint32_t(t) * uint32_t(ld) + chunk : kOutside;
  }
  // scales: lane l has half l % 2 of the four steps of row l / 2 of each 32 (the columns', then the rows')
  const uint8_t* se[kSets];
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int r = 32 * i + (lane >> 1), half = (lane & 1) * 16;
    se[i] = nullptr;
    if (pl.e >= a.E) continue;
    if (r < 16 * NC) {
      if (r < wrows) se[i] = a.qe + (long(pl.e) * a.N + n0 + r) * nb + half;
    } else {
      const int row = r - 16 * NC;
      const int t = row < pl.rows ? token_of(a, pl.row0 + row) : -1;
      if (t >= 0) se[i] = a.pe + long(t) * nb + half;
    }
  }

  v4f acc[NC][NT];
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

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
  // the scales of steps k .. k + 3.  (These loads are not counted by the waits for the
  // stages: with them in flight a wait only takes longer.)
  v4i next[kSets];
  auto fetch = [&](int k) __attribute__((always_inline)) {
    const int at = (s0 + k) * 8;
#pragma unroll
    for (int i = 0; i < kSets; ++i)
      next[i] = load_scales16(se[i] + at, se[i] && k < mine ? nb - at - (lane & 1) * 16 : 0);
  };
  uint8_t* mys = scales + w * kScales;
  auto put = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kSets; ++i) *reinterpret_cast<v4i*>(mys + i * 1024 + lane * 16) = next[i];
  };
  auto multiply = [&](const uint8_t* stage, int k) __attribute__((always_inline)) {
    wait_vm<(S - 1) * L>();
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* sq = stage + w * kStage;
    const uint8_t* sp = sq + 2 * NC * 1024;
    int qe[NC], pe[NT];  // blocks 2 g and 2 g + 1 of the step
#pragma unroll
    for (int i = 0; i < NC; ++i)
      qe[i] = *reinterpret_cast<const uint16_t*>(mys + (i * 16 + m) * 32 + (k & 3) * 8 + 2 * g);
#pragma unroll
    for (int j = 0; j < NT; ++j)
      pe[j] = *reinterpret_cast<const uint16_t*>(mys + ((NC + j) * 16 + m) * 32 + (k & 3) * 8 + 2 * g);
    auto half = [&](auto kk) __attribute__((always_inline)) {
      v4i qf[NC], pf[NT];
      const int slot = ((2 * g + kk) ^ (m & 7)) << 4;
#pragma unroll
      for (int i = 0; i < NC; ++i) qf[i] = *reinterpret_cast<const v4i*>(sq + (i * 16 + m) * 128 + slot);
#pragma unroll
      for (int j = 0; j < NT; ++j) pf[j] = *reinterpret_cast<const v4i*>(sp + (j * 16 + m) * 128 + slot);
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(qf[i]), operand(pf[j]), acc[i][j],
                                                                     kFmtE2M1, kFmtE2M1, kk, qe[i], kk, pe[j]);
    };
    half(std::integral_constant<int, 0>{});
    half(std::integral_constant<int, 1>{});
    // the stage is read before its next loads go out
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  fetch(0);
  issue(st0, 0);
  if constexpr (S == 4) {
    issue(st1, 1);
    issue(st2, 2);
  }
  for (int k = 0; k < mine; k += kGroupSteps) {
    put();  // (the last group's scales are read: multiply ends with a wait for its reads)
    fetch(k + kGroupSteps);
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (S == 2) {
      issue(st1, k + 1); multiply(st0, k);
      issue(st0, k + 2); multiply(st1, k + 1);
      issue(st1, k + 3); multiply(st0, k + 2);
      issue(st0, k + 4); multiply(st1, k + 3);
    } else {
      issue(st3, k + 3); multiply(st0, k);
      issue(st0, k + 4); multiply(st1, k + 1);
      issue(st1, k + 5); multiply(st2, k + 2);
      issue(st2, k + 6); multiply(st3, k + 3);
    }
  }

  stage_barrier();  // every load has landed: the first stage takes the sums
  v4f* part = reinterpret_cast<v4f*>(st0);
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(w * NC * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  // fragment f's sum by wave f % 4: lane l holds columns 4 (l / 16) + 0..3 of row l % 16
  for (int f = w; f < NC * NT; f += kFewWaves) {
    v4f sum = part[f * 64 + lane];
#pragma unroll
    for (int v = 1; v < kFewWaves; ++v) sum += part[(v * NC * NT + f) * 64 + lane];
    const int r = (f % NT) * 16 + m, c = n0 + (f / NT) * 16 + 4 * g;
    if (r >= pl.rows || c >= a.N) continue;
    if (pl.e < a.E && token_of(a, pl.row0 + r) < 0) sum = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    store4(a.out, (long(pl.row0) + r) * a.N + c, sum, a.out_ty);
  }
}

struct TileShape {
  int few, rows, cols;
};

// The tile shape whose launch brings the fewest bytes through a CU: rounds of one
// tile per CU times (rows + columns) of a tile.  The row tiles of ragged groups are
// estimated: groups with a row, each half a tile more than its mean needs.  Among
// equals the first.
TileShape shape_of(const Mx4Args& a, double* cost_of = nullptr) {
  static const TileShape shapes[] = {{1, 16, 64}, {1, 16, 32}, {1, 16, 16}, {1, 32, 32}, {1, 32, 64},
                                     {1, 32, 16}, {1, 64, 64}, {1, 64, 32}, {1, 64, 16}};
  const double groups = a.E * (1.0 - std::exp(-double(a.R) / a.E));  // that are touched
  const double mean = a.R / std::fmax(groups, 1.0);
  TileShape best = shapes[0];
  double least = 1e300;
  for (const TileShape& s : shapes) {
    const double need = mean / s.rows;
    const double rows = a.E == 1 ? std::ceil(a.R / double(s.rows)) : groups * std::fmax(1.0, need + 0.5);
    const double cost = std::ceil(std::ceil(rows) * std::ceil(double(a.N) / s.cols) / kCUs) * (s.rows + s.cols);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  if (cost_of) *cost_of = least;
  return best;
}

long grid_of(const Mx4Args& a, const TileShape& s) {
  return (row_tiles(a, s.rows) * ((a.N + s.cols - 1) / s.cols) + 7) / 8 * 8;
}

// The shape and the workgroups of a launch; false where no launch holds them.
bool plan(const Mx4Args& a, TileShape* s, long* grid) {
  *s = shape_of(a);
  *grid = grid_of(a, *s);
  if (*grid <= max_blocks(kFewWaves * 64)) return true;
  *s = {1, 64, 64};
  *grid = grid_of(a, *s);
  return *grid <= max_blocks(kFewWaves * 64);
}

hipError_t launch_one(const Mx4Args& a, const TileShape& s, long grid, hipStream_t st) {
  if (grid == 0) return hipSuccess;
#define MOE_FEW(NT, NC)                                                                                          \
  case NT * 16 + NC:                                                                                             \
    hipLaunchKernelGGL((k_mx4_few<NC, NT, NT * NC == 1 ? 4 : 2>), dim3(unsigned(grid)), dim3(kFewWaves * 64), 0, \
                       st, a);                                                                                   \
    break;
  switch (s.rows + s.cols / 16) {
    MOE_FEW(1, 1) MOE_FEW(1, 2) MOE_FEW(1, 4)
    MOE_FEW(2, 1) MOE_FEW(2, 2) MOE_FEW(2, 4)
    MOE_FEW(4, 1) MOE_FEW(4, 2) MOE_FEW(4, 4)
  }
#undef MOE_FEW
  return hipGetLastError();
}

}  // namespace

bool mx4_too_large(const Mx4Args& a) {
  TileShape s;
  long grid;
  return !plan(a, &s, &grid);
}

hipError_t launch_mx4(const Mx4Args& a, hipStream_t st, bool* too_large) {
  TileShape s;
  long grid;
  *too_large = !plan(a, &s, &grid);
  return *too_large ? hipSuccess : launch_one(a, s, grid, st);
}

template <int TY, bool GLU>
static hipError_t launch_quant(const uint16_t* x, int R, int K, uint8_t* codes, uint8_t* scales, hipStream_t st) {
  const long chunks = long(R) * K / 8, blocks = (chunks + 256 * kQuantUnroll - 1) / (256 * kQuantUnroll);
  // (a workgroup takes more in turn past 32 per CU)
  hipLaunchKernelGGL((k_quant_mx4<TY, GLU>), dim3(unsigned(blocks < 8192 ? blocks : 8192)), dim3(256), 0, st, x,
                     chunks, K, codes, scales);
  return hipGetLastError();
}

hipError_t launch_quant_mx4(const void* x, int ty, int swiglu, int R, int K, uint8_t* codes, uint8_t* scales,
                            hipStream_t st) {
  if (R == 0) return hipSuccess;
  const uint16_t* xs = static_cast<const uint16_t*>(x);
  if (ty == kBf16)
    return swiglu ? launch_quant<kBf16, true>(xs, R, K, codes, scales, st)
                  : launch_quant<kBf16, false>(xs, R, K, codes, scales, st);
  return swiglu ? launch_quant<kFp16, true>(xs, R, K, codes, scales, st)
                : launch_quant<kFp16, false>(xs, R, K, codes, scales, st);
}

}  // namespace moe
