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
#include "moe_mx4_shape.h"
#include "moe_quant_mx4.h"

namespace moe {
namespace {

// ------------------------------------------------------------------ quantiser
// Eight values a lane, four lanes a block.  Bound by HBM: 2 (SwiGLU: 4) bytes in
// and 17/32 out per value.  4099 rows of 7168: 11.9 to 12.4 us, 6.2 to 6.0 TB/s (four
// chunks of a lane in flight 12.8, and with loads past the caches 14.5).  SwiGLU, 32768 rows of
// 2 x 2048: 70 us, 4.3 TB/s; 488 rows 4.7, a launch.
constexpr int kQuantUnroll = 2;

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
        // (a 32-bit division where it reaches: the 64-bit one costs more than the rest)
        if constexpr (GLU) from += (chunks < (1L << 32) ? long(uint32_t(i) / uint32_t(row_chunks)) : i / row_chunks) * K;
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
    uint64_t lo = 0, hi = 0;
#pragma unroll 1
    for (int i = 0; i < left; ++i) {
      const uint64_t byte = uint64_t(p[i]) << (8 * (i & 7));
      if (i < 8) lo |= byte;
      else hi |= byte;
    }
    v = v4i{int(lo), int(lo >> 32), int(hi), int(hi >> 32)};
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

// A wave makes 16 NC columns by 16 NT rows, its weights' and rows' K steps coming through
// a ring of S stages of its own, so nothing waits for another wave.
//   WK = 4: the four waves of a workgroup have the same columns, and a quarter of the steps
//     each; their sums are added up, in the order of the waves, through LDS.  Where
//     there are too few tiles for the chip.
//   WK = 1: each has columns of its own and all steps.  Where there are many tiles of few
//     rows (a decode batch's experts): nothing to join, and loads that never pause.
// Bound by the weights' bytes.  S is 2, which lets the most workgroups share a CU; but for
// 16 x 16 tiles, which as a rule have a CU to themselves.  (61 tokens, top-8 of 64, us: 7168 ->
// 2048 75 to 83 from process to process, 6.7 to 6.0 TB/s of weights, with four stages 78 and as
// four quarters 113 where these take 75; 2048 -> 7168 84 to 98, 6.0 to 5.1 TB/s.)
constexpr int kFewWaves = 4;

template <int NC, int NT, int S, int WK>
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
  constexpr int kCols = 16 * NC * (kFewWaves / WK);
  const int ncol = (a.N + kCols - 1) / kCols;
  Place pl;
  int ct;
  if (!find_tile(a, 16 * NT, ncol, blockIdx.x, pl, ct)) return;
  const int ld = a.K / 2, nb = a.K / 32;  // bytes of codes and of scales per row of both operands
  const int n0 = ct * kCols + (WK == 1 ? w * 16 * NC : 0);
  if (n0 >= a.N) return;  // (WK = 4: of no wave)
  const int steps = pl.e >= a.E ? 0 : (ld + 127) / 128;
  const int each = (steps + WK - 1) / WK;
  const int s0 = WK == 1 ? 0 : w * each, mine = max(0, min(steps - s0, each));

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

  // fragment (i, j): lane l holds columns 4 (l / 16) + 0..3 of row l % 16
  auto put_out = [&](int i, int j, v4f sum) __attribute__((always_inline)) {
    const int r = j * 16 + m, c = n0 + i * 16 + 4 * g;
    if (r >= pl.rows || c >= a.N) return;
    if (pl.e < a.E && token_of(a, pl.row0 + r) < 0) sum = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    store4(a.out, (long(pl.row0) + r) * a.N + c, sum, a.out_ty);
  };
  if constexpr (WK == 1) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) put_out(i, j, acc[i][j]);
    wait_vm<0>();  // no load is on its way into LDS that another workgroup may get
  } else {
    stage_barrier();  // every load has landed: the first stage takes the sums
    v4f* part = reinterpret_cast<v4f*>(st0);
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j) part[(w * NC * NT + i * NT + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    for (int f = w; f < NC * NT; f += kFewWaves) {  // fragment f's sum by wave f % 4
      v4f sum = part[f * 64 + lane];
#pragma unroll
      for (int v = 1; v < kFewWaves; ++v) sum += part[(v * NC * NT + f) * 64 + lane];
      put_out(f / NT, f % NT, sum);
    }
  }
}

// moe_linear_mx4 for one row: k_mx4_few with the quantiser in front, in every
// workgroup: its lanes quantise the row while the first weights are on their
// way; codes and scales stay in LDS, where all K steps read them.  The codes are the
// quantiser's; sums are put together like those of k_mx4_few with WK = 4, so that a result has
// the bits of the two launches where these take that form (K past 1280, up to 16384 columns).
// Bound by latency, the row's and then the weights' (7168 -> 4096: 7.0 to 8.4 us, quantiser and product by
// themselves 4.8 and 6.6).  Wide products quantise the row in many workgroups, but lose no more than the launch
// saved: 4096 -> 28672 14.3 us, two launches 4.8 + 11.2; 57344 24.5 to 25.1, 4.8 + 20.2; 151936 57.8, 4.8 + 51.1.
constexpr int kOneChunks = 4;  // chunks of 8 values that a lane has
constexpr int kOneMaxK = kOneChunks * kFewWaves * 64 * 8;

template <int XT, bool GLU, int NC>
__global__ __launch_bounds__(kFewWaves * 64) void k_mx4_one(Mx4Args a) {
  constexpr int S = 4, L = 2 * NC, kStage = L * 1024;
  __shared__ __align__(1024) uint8_t st0[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st1[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st2[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t st3[kFewWaves * kStage];
  __shared__ __align__(1024) uint8_t scales[kFewWaves * 1024];
  __shared__ __align__(16) uint8_t codes[kOneMaxK / 2];
  __shared__ __align__(16) uint8_t xscales[kOneMaxK / 32];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  const int ncol = (a.N + 16 * NC - 1) / (16 * NC);
  Place pl;
  int ct;
  if (!find_tile(a, 16, ncol, blockIdx.x, pl, ct)) return;
  const int K = a.K, ld = K / 2, nb = K / 32, n0 = ct * 16 * NC;
  const bool grouped = pl.e < a.E;  // else the row belongs to no group: zeros
  const int steps = grouped ? (ld + 127) / 128 : 0;
  const int each = (steps + kFewWaves - 1) / kFewWaves;
  const int s0 = w * each, mine = max(0, min(steps - s0, each));
  const long wrow = long(grouped ? pl.e : 0) * a.N + n0;
  const uint8_t* wq = static_cast<const uint8_t*>(a.q) + wrow * ld;
  const int wrows = min(16 * NC, a.N - n0);
  const uint32_t wspan = uint32_t(wrows) * uint32_t(ld);
  const int chunk = ((lane & 7) ^ (lane >> 3)) * 16;
  uint32_t ow[L];
#pragma unroll
  for (int i = 0; i < L; ++i) ow[i] = uint32_t(8 * i + (lane >> 3)) * uint32_t(ld) + chunk;
  auto issue = [&](uint8_t* stage, int k) __attribute__((always_inline)) {
    const int at = (s0 + k) * 128;
    const bool in = k < mine && chunk < ld - at;
#pragma unroll
    for (int i = 0; i < L; ++i) dma16<true>(wq, wspan, in ? ow[i] + at : kOutside, stage + w * kStage + i * 1024);
  };
  // the weights' scales, four steps at a time: as in k_mx4_few
  const uint8_t* se = (lane >> 1) < wrows && grouped ? a.qe + (wrow + (lane >> 1)) * nb + (lane & 1) * 16 : nullptr;
  v4i next;
  auto fetch = [&](int k) __attribute__((always_inline)) {
    const int at = (s0 + k) * 8;
    next = load_scales16(se + at, se && k < mine ? nb - at - (lane & 1) * 16 : 0);
  };
  uint8_t* mys = scales + w * 1024;

  // the row comes in ahead of the first weights; one that names no token is zeros
  const int t = grouped ? token_of(a, pl.row0) : -1;
  const uint16_t* x = static_cast<const uint16_t*>(a.p) + long(max(t, 0)) * (GLU ? 2L * K : K);
  quant_raw8 raw[kOneChunks][GLU ? 2 : 1];
#pragma unroll
  for (int i = 0; i < kOneChunks; ++i) {
    const int c = (i * kFewWaves * 64 + int(threadIdx.x)) * 8;
#pragma unroll
    for (int h = 0; h < (GLU ? 2 : 1); ++h)
      raw[i][h] = t >= 0 && c < K ? *reinterpret_cast<const quant_raw8*>(x + h * K + c) : quant_raw8{0, 0, 0, 0};
  }
  fetch(0);
  __builtin_amdgcn_sched_barrier(0);
  issue(st0, 0);
  issue(st1, 1);
  issue(st2, 2);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kOneChunks; ++i) {
    const int c = (i * kFewWaves * 64 + int(threadIdx.x)) * 8;
    const f8v v = quant_value8<XT, GLU>(raw[i][0], raw[i][GLU ? 1 : 0]);
    const uint32_t scale = mx4_scale(group_top_dpp(quant_top8(v), 4));
    // the last step's columns past K are zeros
    if (c < (K + 255) / 256 * 256) {
      *reinterpret_cast<uint32_t*>(codes + c / 2) = mx4_codes8(v, scale);
      if (c % 32 == 0) xscales[c / 32] = uint8_t(scale);
    }
  }
  lds_barrier();

  v4f acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](const uint8_t* stage, int k) __attribute__((always_inline)) {
    wait_vm<(S - 1) * L>();
    __builtin_amdgcn_sched_barrier(0);
    const bool has = m == 0 && k < mine;
    const int pe = has ? *reinterpret_cast<const uint16_t*>(xscales + (s0 + k) * 8 + 2 * g) : 0;
    int qe[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i)
      qe[i] = *reinterpret_cast<const uint16_t*>(mys + (i * 16 + m) * 32 + (k & 3) * 8 + 2 * g);
    auto half = [&](auto kk) __attribute__((always_inline)) {
      v4i pf = {0, 0, 0, 0};
      if (has) pf = *reinterpret_cast<const v4i*>(codes + (s0 + k) * 128 + (2 * g + kk) * 16);
      const int slot = ((2 * g + kk) ^ (m & 7)) << 4;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const v4i qf = *reinterpret_cast<const v4i*>(stage + w * kStage + (i * 16 + m) * 128 + slot);
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(operand(qf), operand(pf), acc[i], kFmtE2M1, kFmtE2M1, kk,
                                                                qe[i], kk, pe);
      }
    };
    half(std::integral_constant<int, 0>{});
    half(std::integral_constant<int, 1>{});
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_waitcnt(0xC07F);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  for (int k = 0; k < mine; k += kGroupSteps) {
    *reinterpret_cast<v4i*>(mys + lane * 16) = next;
    fetch(k + kGroupSteps);
    __builtin_amdgcn_sched_barrier(0);
    issue(st3, k + 3); multiply(st0, k);
    issue(st0, k + 4); multiply(st1, k + 1);
    issue(st1, k + 5); multiply(st2, k + 2);
    issue(st2, k + 6); multiply(st3, k + 3);
  }
  stage_barrier();  // every load has landed: the first stage takes the sums
  v4f* part = reinterpret_cast<v4f*>(st0);
#pragma unroll
  for (int i = 0; i < NC; ++i) part[(w * NC + i) * 64 + lane] = acc[i];
  __syncthreads();
  if (w < NC && m == 0) {  // fragment w: lane l holds columns 4 (l / 16) + 0..3 of row l % 16
    v4f sum = part[w * 64 + lane];
#pragma unroll
    for (int u = 1; u < kFewWaves; ++u) sum += part[(u * NC + w) * 64 + lane];
    const int c = n0 + w * 16 + 4 * g;
    if (c < a.N) store4(a.out, long(pl.row0) * a.N + c, t < 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : sum, a.out_ty);
  }
}

// Where there are tiles enough: 256 columns by BM rows per workgroup, four waves of
// BM / 2 rows by 128 columns each, so that a wave reads every fragment for four
// instructions and a SIMD's registers hold one wave's sums.  Two stages of a K
// step; a step's loads go out when all have read the stage before them, in the
// middle of a step, and are needed a step later.
//
// The 32 x 32 x 64 instruction it is built from issues at twice the rate of the 16 x
// 16 x 128 one on 4-bit operands (9.7 PFLOP/s against 4.9, nothing else running).
//
// Bound by power and the loads into LDS: a step of 256 rows takes 3050 clocks, its matrix
// instructions 2048 (without its loads 2350, without the instructions 2740), at 1.5 to 1.8 GHz.
// 4096 x 4096 x 7168: 60 to 62 us, 4.0 PFLOP/s; 32768 rows of 64 groups, 4096 -> 1536: 155 to 168 from process to
// process, 2.7 to 2.5 (with the tiles in blocks across groups 165 where these take 160, 427 MB from memory and
// the last cache in the place of 322; 2048 -> 7168 402 in the place of 414; tiles of up to 128 rows in code of
// their own, and these last: the same).
constexpr int kThreads = 256;
constexpr int kBN = kMx4Cols;

typedef float v16f __attribute__((ext_vector_type(16)));

// The stream of ROWS rows of an operand over the K steps, in 1 KB wave loads.
template <int ROWS>
struct Rows {
  static constexpr int kBytes = ROWS * 128;
  static constexpr int kLoads = kBytes / 1024 / (kThreads / 64);
  const uint8_t* base;
  long left;  // bytes from base to the end of what may be read
  uint32_t off[kLoads];
  int chunk;  // byte of the lane's chunk in the 128-byte step

  // `index`: the memory row of each of the tile's nindex rows, counted from b; one
  // outside [0, nrows) reads as zeros.
  __device__ __forceinline__ void init(const uint8_t* b, long bytes, int ld, int w, int lane, const int32_t* index,
                                       int nindex, int nrows) {
    base = b;
    left = bytes;
    chunk = ((lane & 7) ^ (lane >> 3)) * 16;  // chunk c of row r lies in slot c ^ (r & 7)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int row = (w * kLoads + i) * 8 + (lane >> 3);
      if (index) {
        const int t = row < nindex ? index[row] : -1;
        off[i] = t >= 0 && t < nrows ? uint32_t(t) * uint32_t(ld) + chunk : kOutside;
      } else {
        off[i] = uint32_t(row) * uint32_t(ld) + chunk;
      }
    }
  }
  // kleft: bytes of a row from this step on; chunks past them read as zeros
  __device__ __forceinline__ void issue(uint8_t* stage, int w, int kleft) {
    const uint32_t n = uint32_t(left < 0 ? 0L : left > 0x7FFFFFFFL ? 0x7FFFFFFFL : left);
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      dma16<false>(base, n, chunk < kleft ? off[i] : kOutside, stage + (w * kLoads + i) * 1024);
    base += 128;
    left -= 128;
  }
};

template <int BM>
__global__ __launch_bounds__(kThreads, 1) void k_mx4(Mx4Args a) {
  constexpr int NF = 4, MF = BM / 64;  // fragments of 32 columns and rows of a wave
  using PS = Rows<BM>;
  using QS = Rows<kBN>;
  __shared__ __align__(1024) uint8_t p0[PS::kBytes];
  __shared__ __align__(1024) uint8_t p1[PS::kBytes];
  __shared__ __align__(1024) uint8_t q0[QS::kBytes];
  __shared__ __align__(1024) uint8_t q1[QS::kBytes];
  // scales of four steps, 32 bytes of each row (the columns', then the rows'): eight of
  // step s at unit s ^ (row >> 3 & 3), so that the 32 rows of a read spread over the banks
  __shared__ __align__(1024) uint8_t sc[2 * (kBN + BM) * 32];

  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = w >> 1, wn = w & 1;
  const int ncol = (a.N + kBN - 1) / kBN, ld = a.K / 2, nb = a.K / 32;
  Place pl;
  int ct;
  if (!find_tile<true>(a, BM, ncol, blockIdx.x, pl, ct)) return;
  // (one tile of the whole workgroup: its numbers stay in scalar registers)
  pl.e = __builtin_amdgcn_readfirstlane(pl.e);
  pl.row0 = __builtin_amdgcn_readfirstlane(pl.row0);
  pl.rows = __builtin_amdgcn_readfirstlane(pl.rows);
  ct = __builtin_amdgcn_readfirstlane(ct);
  const bool grouped = pl.e < a.E;
  const int n0 = ct * kBN, steps = grouped ? (ld + 127) / 128 : 0;
  const long wrow = long(pl.e) * a.N + n0;
  // The first loads go out as early as they can: the columns', then, with the rows'
  // places known, the rows'.
  QS qs;
  qs.init(static_cast<const uint8_t*>(a.q) + wrow * ld, grouped ? long(min(kBN, a.N - n0)) * ld : 0, ld, w, lane,
          nullptr, 0, 0);
  qs.issue(q0, w, ld);
  PS ps;
  const uint8_t* P = static_cast<const uint8_t*>(a.p);
  if (a.row_token) ps.init(P, grouped ? long(a.T) * ld : 0, ld, w, lane, a.row_token + pl.row0, pl.rows, a.T);
  else ps.init(P + long(pl.row0) * ld, grouped ? long(pl.rows) * ld : 0, ld, w, lane, nullptr, 0, 0);
  // scales: two lanes have a row's 32 bytes, lane l half l % 2 of row l / 2 of a wave's 32
  constexpr int kSets = (kBN + BM) / 128;
  const uint8_t* se[kSets];
#pragma unroll
  for (int i = 0; i < kSets; ++i) {
    const int r = i * 128 + w * 32 + (lane >> 1), part = (lane & 1) * 16;
    se[i] = nullptr;
    if (!grouped) continue;
    if (i < 2) {
      if (n0 + r < a.N) se[i] = a.qe + (wrow + r) * nb + part;
    } else if (r - kBN < pl.rows) {
      const int t = token_of(a, pl.row0 + r - kBN);
      if (t >= 0) se[i] = a.pe + long(t) * nb + part;
    }
  }
  ps.issue(p0, w, ld);
  v4i next[kSets];
  auto fetch = [&](int s) __attribute__((always_inline)) {  // of steps s .. s + 3
    const int at = s * 8, left = nb - at - (lane & 1) * 16;
#pragma unroll
    for (int i = 0; i < kSets; ++i) next[i] = load_scales16(se[i] + at, se[i] ? left : 0);
  };
  auto put = [&](uint8_t* s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kSets; ++i) {
      const int r = i * 128 + w * 32 + (lane >> 1), part = (lane & 1) * 16, x = (r >> 3 & 3) * 8;
      uint8_t* to = s + r * 32;
      *reinterpret_cast<int2*>(to + (part ^ x)) = make_int2(next[i][0], next[i][1]);
      *reinterpret_cast<int2*>(to + ((part + 8) ^ x)) = make_int2(next[i][2], next[i][3]);
    }
  };

  v16f acc[NF][MF];
#pragma unroll
  for (int i = 0; i < NF; ++i)
#pragma unroll
    for (int j = 0; j < MF; ++j)
#pragma unroll
      for (int u = 0; u < 16; ++u) acc[i][j][u] = 0.0f;

  int kleft = ld - 128;  // bytes of a row from the next step to load on
  auto issue = [&](uint8_t* sp, uint8_t* sq) __attribute__((always_inline)) {
    ps.issue(sp, w, kleft);
    qs.issue(sq, w, kleft);
    kleft -= 128;
  };
  // A quarter of a step: of each row's eight blocks, lane l of row l % 32 has blocks 4 (l /
  // 32) + 0..3, one of them in each quarter; their scales are one word.  Each
  // quarter is read while the one before it is multiplied.
  const int r32 = lane & 31, h = lane >> 5;
  struct Quarter {
    v4i q[NF], p[MF];
  };
  struct Scales {
    int q[NF], p[MF];
  };
  auto read = [&](Quarter& f, const uint8_t* sp, const uint8_t* sq, int b) __attribute__((always_inline)) {
    const int slot = ((4 * h + b) ^ (r32 & 7)) << 4;
#pragma unroll
    for (int i = 0; i < NF; ++i)
      f.q[i] = *reinterpret_cast<const v4i*>(sq + ((wn * NF + i) * 32 + r32) * 128 + slot);
#pragma unroll
    for (int i = 0; i < MF; ++i)
      f.p[i] = *reinterpret_cast<const v4i*>(sp + ((wm * MF + i) * 32 + r32) * 128 + slot);
  };
  auto read_scales = [&](Scales& f, const uint8_t* s, int step) __attribute__((always_inline)) {
    const int at = (((step & 3) ^ (r32 >> 3 & 3)) << 3) + 4 * h;
#pragma unroll
    for (int i = 0; i < NF; ++i) f.q[i] = *reinterpret_cast<const int*>(s + ((wn * NF + i) * 32 + r32) * 32 + at);
#pragma unroll
    for (int i = 0; i < MF; ++i)
      f.p[i] = *reinterpret_cast<const int*>(s + (kBN + (wm * MF + i) * 32 + r32) * 32 + at);
  };
  auto multiply = [&](const Quarter& f, const Scales& e, auto b) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(operand(f.q[i]), operand(f.p[j]), acc[i][j],
                                                                  kFmtE2M1, kFmtE2M1, b, e.q[i], b, e.p[j]);
  };
  auto spread = [&]() __attribute__((always_inline)) {  // reads between the products
#pragma unroll
    for (int i = 0; i < NF + MF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, NF * MF / (NF + MF), 0);
    }
  };
  // The products before this point stay before it: the compiler would else move those of
  // a whole step behind the branches of fetch, where nothing overlaps them.
  auto hold = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NF; ++i)
#pragma unroll
      for (int j = 0; j < MF; ++j) asm volatile("" : "+a"(acc[i][j]));
  };
  Quarter f0, f1;
  Scales now, then;
  // Step s from stage x, with y the next stage; the next step's scales are in `sc`.
  // (what is read from y after the last step goes unused)
  auto step = [&](uint8_t* px, uint8_t* qx, const uint8_t* py, const uint8_t* qy, const uint8_t* sc, int s)
                  __attribute__((always_inline)) {
    read(f1, px, qx, 1);
    multiply(f0, now, std::integral_constant<int, 0>{});
    spread();
    read(f0, px, qx, 2);
    multiply(f1, now, std::integral_constant<int, 1>{});
    spread();
    read(f1, px, qx, 3);
    multiply(f0, now, std::integral_constant<int, 2>{});
    spread();
    hold();
    stage_barrier();  // stage x is read, stage y has arrived
    issue(px, qx);
    read(f0, py, qy, 0);
    read_scales(then, sc, s + 1);
    multiply(f1, now, std::integral_constant<int, 3>{});
#pragma unroll
    for (int i = 0; i < NF * MF; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    }
    hold();
    now = then;
  };
  // The next four steps' scales are fetched beside the loads of every fourth step, which
  // the step behind it waits for anyway, and lie in LDS a barrier before they are read.
  constexpr int kGroup = (kBN + BM) * 32;
  auto scales_of = [&](int s) __attribute__((always_inline)) { return sc + (s / kGroupSteps & 1) * kGroup; };
  if (steps) {
    fetch(0);
    issue(p1, q1);
    put(sc);
    stage_barrier_but<PS::kLoads + QS::kLoads>();
    read(f0, p0, q0, 0);
    read_scales(now, sc, 0);
    for (int s = 0; s < steps; s += 2) {
      const bool first = s % kGroupSteps == 0;  // of four
      step(p0, q0, p1, q1, scales_of(s + 1), s);
      if (first) fetch(s + kGroupSteps);
      // (an odd last step is made up with one of zeros: a branch here would cost the sums their registers)
      step(p1, q1, p0, q0, scales_of(s + 2), s + 1);
      if (first) put(scales_of(s + kGroupSteps));
    }
  }

  // Lane l holds columns 8 b + 4 (l / 32) + 0..3 (b = 0..3) of row l % 32 of each
  // fragment.  32 rows at a time go through a piece of LDS of the wave's own, so that
  // a store covers whole rows of its 128 columns.
  stage_barrier();  // no stage is read or filled any more
  int el = lane;
  asm volatile("" : "+v"(el));  // addresses from here on are not formed before the loop, which has no registers for them
  const int row = el & 31, eh = el >> 5;
  const int r0 = wm * (BM / 2), c0 = n0 + wn * 128;
  uint8_t* piece = (w & 2 ? q1 : q0) + (w & 1) * 16384;
  auto put_out = [&](auto ty) __attribute__((always_inline)) {
    constexpr int TY = decltype(ty)::value, kEl = TY == kFp32 ? 4 : 2;
    constexpr int kAcross = 128 * kEl / 16, kDown = 64 / kAcross;  // 16-byte chunks of a row, rows of a store
    uint8_t* rows0 = static_cast<uint8_t*>(a.out) + (long(pl.row0) + r0) * a.N * kEl;
#pragma unroll
    for (int j = 0; j < MF; ++j) {
      const int r = r0 + j * 32 + row;
      const bool dead = a.row_token && grouped && r < pl.rows && token_of(a, pl.row0 + r) < 0;
#pragma unroll
      for (int i = 0; i < NF; ++i)
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          v4f v = {acc[i][j][4 * b], acc[i][j][4 * b + 1], acc[i][j][4 * b + 2], acc[i][j][4 * b + 3]};
          if (dead) v = v4f{0.0f, 0.0f, 0.0f, 0.0f};
          const int unit = i * 8 + b * 2 + eh;  // four columns
          if constexpr (TY == kFp32)
            *reinterpret_cast<v4f*>(piece + row * 512 + ((unit ^ row) << 4)) = v;
          else
            *reinterpret_cast<uint2*>(piece + row * 256 + (((unit >> 1) ^ (row & 15)) << 4) + (unit & 1) * 8) = round4(v, TY);
        }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int u = 0; u < 32 / kDown; ++u) {
        const int rr = u * kDown + el / kAcross, ch = el % kAcross;
        const v4i d = *reinterpret_cast<const v4i*>(piece + rr * (kAcross * 16) + ((ch ^ (rr % kAcross)) << 4));
        const int at = j * 32 + rr, c = c0 + ch * (16 / kEl);
        store16(rows0, d, r0 + at < pl.rows && c < a.N ? uint32_t(at * a.N + c) * kEl : kOutside);
      }
      __builtin_amdgcn_wave_barrier();
    }
  };
  if (a.out_ty == kFp32) put_out(std::integral_constant<int, kFp32>{});
  else if (a.out_ty == kFp16) put_out(std::integral_constant<int, kFp16>{});
  else put_out(std::integral_constant<int, kBf16>{});
}

long grid_of(const Mx4Args& a, const Mx4Shape& s) {
  return (row_tiles(a, s.rows) * ((a.N + s.cols - 1) / s.cols) + 7) / 8 * 8;
}

// The shape and the workgroups of a launch; false where no launch holds them.
bool plan(const Mx4Args& a, Mx4Shape* s, long* grid) {
  *s = mx4_shape(a.R, a.N, a.K, a.E);
  *grid = grid_of(a, *s);
  if (*grid <= max_blocks(kThreads)) return true;
  *s = {kMx4Big, 256, kBN};
  *grid = grid_of(a, *s);
  return *grid <= max_blocks(kThreads);
}

hipError_t launch_one(const Mx4Args& a, const Mx4Shape& s, long grid, hipStream_t st) {
  static_assert(kThreads == kFewWaves * 64, "one limit of a launch");
  if (grid == 0) return hipSuccess;
  if (s.kind == kMx4Big) {
    if (s.rows == 256) hipLaunchKernelGGL((k_mx4<256>), dim3(unsigned(grid)), dim3(kThreads), 0, st, a);
    else hipLaunchKernelGGL((k_mx4<128>), dim3(unsigned(grid)), dim3(kThreads), 0, st, a);
    return hipGetLastError();
  }
#define MOE_FEW(NC, NT, S, WK) \
  hipLaunchKernelGGL((k_mx4_few<NC, NT, S, WK>), dim3(unsigned(grid)), dim3(kThreads), 0, st, a)
  if (s.kind == kMx4Rows) {
    switch (s.rows + s.cols / 64) {
      case 17: MOE_FEW(1, 1, 2, 1); break;
      case 18: MOE_FEW(2, 1, 2, 1); break;
      case 20: MOE_FEW(4, 1, 2, 1); break;
      case 34: MOE_FEW(2, 2, 2, 1); break;
      case 36: MOE_FEW(4, 2, 2, 1); break;
      case 66: MOE_FEW(2, 4, 2, 1); break;
    }
    return hipGetLastError();
  }
  switch (s.rows + s.cols / 16) {
    case 17: MOE_FEW(1, 1, 4, 4); break;
    case 18: MOE_FEW(2, 1, 2, 4); break;
    case 20: MOE_FEW(4, 1, 2, 4); break;
    case 33: MOE_FEW(1, 2, 2, 4); break;
    case 34: MOE_FEW(2, 2, 2, 4); break;
    case 36: MOE_FEW(4, 2, 2, 4); break;
    case 65: MOE_FEW(1, 4, 2, 4); break;
    case 66: MOE_FEW(2, 4, 2, 4); break;
    case 68: MOE_FEW(4, 4, 2, 4); break;
  }
#undef MOE_FEW
  return hipGetLastError();
}

}  // namespace

bool mx4_too_large(const Mx4Args& a) {
  Mx4Shape s;
  long grid;
  return !plan(a, &s, &grid);
}

hipError_t launch_mx4(const Mx4Args& a, hipStream_t st, bool* too_large) {
  Mx4Shape s, ts;
  long grid, tail_grid;
  *too_large = !plan(a, &s, &grid);
  if (*too_large) return hipSuccess;
  const int rows = a.offsets ? a.R : mx4_first_rows(a.R, a.N, a.K);
  if (rows == a.R) return launch_one(a, s, grid, st);
  Mx4Args head = a, tail = a;
  head.R = rows;
  tail.R = a.R - rows;
  tail.out = static_cast<uint8_t*>(a.out) + long(rows) * a.N * (a.out_ty == kFp32 ? 4 : 2);
  if (a.row_token) {
    tail.row_token = a.row_token + rows;
  } else {
    tail.p = static_cast<const uint8_t*>(a.p) + long(rows) * (a.K / 2);
    tail.pe = a.pe + long(rows) * (a.K / 32);
  }
  *too_large = !plan(head, &s, &grid) || !plan(tail, &ts, &tail_grid);
  if (*too_large) return hipSuccess;
  const hipError_t e = launch_one(head, s, grid, st);
  return e != hipSuccess ? e : launch_one(tail, ts, tail_grid, st);
}

bool linear_mx4_is_one_launch(int R, int K) { return R <= 1 && K <= kOneMaxK; }

hipError_t launch_linear_mx4_one(const Mx4Args& a, int x_ty, int swiglu, hipStream_t st) {
  // columns per workgroup: the fewest bytes through a CU
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
#define MOE_ONE(XT, GLU, NC) hipLaunchKernelGGL((k_mx4_one<XT, GLU, NC>), dim3(grid), dim3(kFewWaves * 64), 0, st, a)
#define MOE_ONE_NC(XT, GLU)           \
  do {                                \
    if (nc == 2) MOE_ONE(XT, GLU, 2); \
    else MOE_ONE(XT, GLU, 1);         \
  } while (0)
  if (x_ty == kBf16) {
    if (swiglu) MOE_ONE_NC(kBf16, true);
    else MOE_ONE_NC(kBf16, false);
  } else {
    if (swiglu) MOE_ONE_NC(kFp16, true);
    else MOE_ONE_NC(kFp16, false);
  }
#undef MOE_ONE_NC
#undef MOE_ONE
  return hipGetLastError();
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
