// moe_norm.hip -- root-mean-square norm of 16-bit rows with the residual's
// addition, its quantised forms and its gradients.
//
//   s = x + residual (rounded to the rows' type: it is what the residual stream
//   carries on), rstd = 1 / sqrt(mean(s^2) + eps), y = s * rstd * weight.
//   With n = s * rstd, g = dy * weight:
//   dx = rstd * (g - n * mean(g * n)) + dsum, dweight = sum over rows of dy * n.
//
// One pass over the data either way: a row's values stay in registers between
// its sum and its result, and the backward pass adds a row up for dweight while
// it has it for dx.  All sums are fp32; y is rounded once, to 16 bits or to the
// codes, which are made from the fp32 value.
#include "moe_norm.h"

#include "moe_quant_mx4.h"

namespace moe {
namespace {

template <int TY>
__device__ __forceinline__ quant_raw8 narrow8(const f8v& v) {
  if constexpr (TY == kBf16) return __builtin_bit_cast(quant_raw8, __builtin_convertvector(v, bf8v));
  else return __builtin_bit_cast(quant_raw8, __builtin_convertvector(v, h8v));
}

// The values as rounded to fp32: a product is else rounded once, straight to fp16,
// where nothing but that is made of it, and y would depend on what is asked for beside it.
__device__ __forceinline__ void hold(f8v& v) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float f = v[j];
    asm volatile("" : "+v"(f));
    v[j] = f;
  }
}

__device__ __forceinline__ quant_raw8 load8(const void* p, long at) {
  return *reinterpret_cast<const quant_raw8*>(static_cast<const uint16_t*>(p) + at);
}
__device__ __forceinline__ void store8(void* p, long at, const quant_raw8& v) {
  *reinterpret_cast<quant_raw8*>(static_cast<uint16_t*>(p) + at) = v;
}
// the same past the caches
__device__ __forceinline__ void store8_late(void* p, long at, const quant_raw8& v) {
  __builtin_nontemporal_store(v, reinterpret_cast<quant_raw8*>(static_cast<uint16_t*>(p) + at));
}

// eight floats at a 16-byte aligned address
__device__ __forceinline__ f8v load8f(const float* p) {
  const v4f a = *reinterpret_cast<const v4f*>(p), b = *reinterpret_cast<const v4f*>(p + 4);
  return f8v{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ void store8f(float* p, const f8v& v) {
  *reinterpret_cast<v4f*>(p) = v4f{v[0], v[1], v[2], v[3]};
  *reinterpret_cast<v4f*>(p + 4) = v4f{v[4], v[5], v[6], v[7]};
}

// eight weights, 16-bit (TY) or fp32
template <int TY>
__device__ __forceinline__ f8v weight8(const void* w, int fp32, int c) {
  if (fp32) return load8f(static_cast<const float*>(w) + c);
  return quant_widen8<TY>(load8(w, c));
}

// The sum over a wave, in every lane: within 16 lanes by DPP, then the four rows'.
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_f32<0xB1>(v);
  v += dpp_f32<0x4E>(v);
  v += dpp_f32<0x141>(v);
  v += dpp_f32<0x140>(v);
  const int b = __float_as_int(v);
  const float p = __int_as_float(__builtin_amdgcn_readlane(b, 0)), q = __int_as_float(__builtin_amdgcn_readlane(b, 16));
  const float r = __int_as_float(__builtin_amdgcn_readlane(b, 32)), s = __int_as_float(__builtin_amdgcn_readlane(b, 48));
  return (p + q) + (r + s);
}
__device__ __forceinline__ uint32_t wave_top(uint32_t v) {
  v = group_top_dpp(v, 16);
  const uint32_t p = __builtin_amdgcn_readlane(v, 0), q = __builtin_amdgcn_readlane(v, 16);
  const uint32_t r = __builtin_amdgcn_readlane(v, 32), s = __builtin_amdgcn_readlane(v, 48);
  return max(max(p, q), max(r, s));
}

// The same over a row's THREADS lanes; `slot`: LDS of the row's own for this one use.
template <int THREADS>
__device__ __forceinline__ float row_sum(float v, float* slot) {
  v = wave_sum(v);
  if constexpr (THREADS > kWave) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) v += slot[i];
  }
  return v;
}
template <int THREADS>
__device__ __forceinline__ uint32_t row_top(uint32_t v, uint32_t* slot) {
  v = wave_top(v);
  if constexpr (THREADS > kWave) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int i = 0; i < THREADS / kWave; ++i) v = max(v, slot[i]);
  }
  return v;
}

constexpr float kTiny = 0x1p-80f;  // keeps the squares of any finite row's values, and their sum, inside fp32

// THREADS lanes per row (64: four rows per workgroup), NC chunks of 8 values a lane.
// Bound by HBM: 8 bytes a value with the residual, 16384 rows of 4096: 85 to 93 us from process to
// process, 6.3 to 5.8 TB/s; to int8 codes 83, 5.7, to MXFP4 78, 5.6 (7 and 6.5 bytes a value).
//
// Beside codes the sum is stored past the caches, as it is next read when the layer's result is
// there (4099 rows of 4096 to e4m3: 21 to 25 us, 28 through them where these take 25).  By itself it is not: in front of its own
// gradients 16384 rows of 4096 take 85 us, 96 past the caches.
template <int TY, int FMT, int THREADS, int NC>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void k_norm(NormArgs a) {
  constexpr int kRows = THREADS < 256 ? 256 / THREADS : 1;
  __shared__ float s_sum[THREADS / kWave], s_again[THREADS / kWave];
  __shared__ uint32_t s_top[THREADS / kWave];
  const int tid = threadIdx.x % THREADS, K = a.K;
  const long row = long(blockIdx.x) * kRows + threadIdx.x / THREADS;
  const bool some = row < a.R;
  f8v v[NC], w[NC];
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * THREADS + tid) * 8;
    v[i] = f8v{};
    w[i] = f8v{};
    if (some && c < K) {
      v[i] = quant_widen8<TY>(load8(a.x, row * K + c));
      if (a.res) {
        const quant_raw8 s = narrow8<TY>(v[i] + quant_widen8<TY>(load8(a.res, row * K + c)));
        if (a.sum) {
          if constexpr (FMT == kQNone) store8(a.sum, row * K + c, s);
          else store8_late(a.sum, row * K + c, s);
        }
        v[i] = quant_widen8<TY>(s);
      }
      w[i] = weight8<TY>(a.weight, a.weight_fp32, c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  ss = row_sum<THREADS>(ss, s_sum);
  float unit = 1.0f, eps = a.eps;
  if (!(ss < __builtin_inff())) {
    // squares past fp32's range: again with the row scaled down (a row that holds an
    // infinity or NaN comes out as the formula has it)
    unit = kTiny;
    eps *= kTiny * kTiny;
    ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      v[i] *= kTiny;
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(v[i][j], v[i][j], ss);
    }
    ss = row_sum<THREADS>(ss, s_again);
  }
  const float rstd = 1.0f / sqrtf(ss / float(K) + eps);
  if (a.rstd && some && tid == 0) a.rstd[row] = rstd * unit;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * THREADS + tid) * 8;
    v[i] = v[i] * rstd * w[i];
    if constexpr (TY == kFp16) hold(v[i]);
    if (a.y && some && c < K) store8(a.y, row * K + c, narrow8<TY>(v[i]));
  }
  if constexpr (FMT == kQI8) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < NC; ++i) top = max(top, quant_top8(v[i]));
    const QuantScale q = quant_scale(row_top<THREADS>(top, s_top));
    if (!some) return;
    if (tid == 0) static_cast<float*>(a.scales)[row] = q.scale;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      if (c < K) *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.codes) + row * K + c) = quant_codes8(v[i], q);
    }
  }
  if constexpr (FMT == kQE4M3) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      const uint32_t top = group_top_dpp(quant_top8(v[i]), a.group / 8);  // 4 or 16 lanes
      const bool finite = top < 0x7F800000u;
      const float mult = quant_mult(__uint_as_float(finite ? top : 0u));
      uint2 q = make_uint2(0, 0);
      if (finite) {
        const f8v u = v[i] * mult;
        q = make_uint2(enc_e4m3x4(u[0], u[1], u[2], u[3]), enc_e4m3x4(u[4], u[5], u[6], u[7]));
      }
      if (some && c < K) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(a.codes) + row * K + c) = q;
        if (c % a.group == 0)
          static_cast<float*>(a.scales)[row * (K / a.group) + c / a.group] =
              finite ? 1.0f / mult : __uint_as_float(0x7FC00000u);
      }
    }
  }
  if constexpr (FMT == kQMx4) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      const uint32_t scale = mx4_scale(group_top_dpp(quant_top8(v[i]), 4));
      const uint32_t q = mx4_codes8(v[i], scale);
      if (some && c < K) {
        *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(a.codes) + row * (K / 2) + c / 2) = q;
        if (c % 32 == 0) static_cast<uint8_t*>(a.scales)[row * (K / 32) + c / 32] = uint8_t(scale);
      }
    }
  }
}

// ------------------------------------------------------------------ gradients
// Workgroups of the backward pass; each takes every so-many-th row and keeps
// its part of dweight in registers.
// (us, 16384 rows of 4096: 512 of 256 lanes 104, 512 of 512 105, 256 of 1024 102; 4099 of 7168: 57, 52,
// 50; 1024 of 4096: 16.5, 15.7, 14.1; twice as many are slower everywhere.)
int grad_rows(int K) { return K <= 1024 ? 4 : 1; }  // rows a workgroup has at a time
int grad_blocks(int R, int K) {
  const int n = grad_rows(K), most = K <= 2048 ? 512 : 256;
  const long need = (long(R) + n - 1) / n;
  return int(need < most ? need : most);
}

// Bound by HBM: 8 bytes a value with the sum's gradient; 16384 rows of 4096: 97 to 111 us from process
// to process and 5 for the join, 5.3 to 4.6 TB/s.
template <int TY, int THREADS, int NC>
__global__ __launch_bounds__(THREADS < 256 ? 256 : THREADS) void k_norm_grad(NormGradArgs a) {
  constexpr int kRows = THREADS < 256 ? 256 / THREADS : 1;
  __shared__ float s_sum[2][THREADS / kWave];
  __shared__ __align__(16) float s_dw[kRows > 1 ? kRows * NC * THREADS * 8 : 4];
  const int tid = threadIdx.x % THREADS, sub = threadIdx.x / THREADS, K = a.K;
  f8v w[NC], dw[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * THREADS + tid) * 8;
    w[i] = c < K ? weight8<TY>(a.weight, a.weight_fp32, c) : f8v{};
    dw[i] = f8v{};
  }
  const float inv = 1.0f / float(K);
  int turn = 0;
  for (long r0 = long(blockIdx.x) * kRows; r0 < a.R; r0 += long(gridDim.x) * kRows) {
    const long row = r0 + sub;
    const bool some = row < a.R;
    const float rstd = some ? a.rstd[row] : 0.0f;
    f8v n[NC], dy[NC];
    quant_raw8 ds[NC];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      n[i] = f8v{};
      dy[i] = f8v{};
      ds[i] = quant_raw8{0, 0, 0, 0};
      if (some && c < K) {
        n[i] = quant_widen8<TY>(load8(a.sum, row * K + c)) * rstd;
        dy[i] = quant_widen8<TY>(load8(a.dy, row * K + c));
        if (a.dsum) ds[i] = load8(a.dsum, row * K + c);
      }
      const f8v gn = dy[i] * w[i] * n[i];
#pragma unroll
      for (int j = 0; j < 8; ++j) sum += gn[j];
    }
    sum = row_sum<THREADS>(sum, s_sum[turn]) * inv;
    turn ^= 1;  // (a wave is at most one row ahead of the others)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      dw[i] += dy[i] * n[i];
      if (a.dx && some && c < K) {
        f8v dx = (dy[i] * w[i] - n[i] * sum) * rstd;
        if (a.dsum) dx += quant_widen8<TY>(ds[i]);
        store8(a.dx, row * K + c, narrow8<TY>(dx));
      }
    }
  }
  if (!a.dw) return;
  float* part = a.partial + long(blockIdx.x) * K;
  if constexpr (kRows > 1) {
#pragma unroll
    for (int i = 0; i < NC; ++i) store8f(s_dw + ((sub * NC + i) * THREADS + tid) * 8, dw[i]);
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int u = 1; u < kRows; ++u) dw[i] += load8f(s_dw + ((u * NC + i) * THREADS + tid) * 8);
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (i * THREADS + tid) * 8;
    if (c < K) store8f(part + c, dw[i]);
  }
}

// dweight = the workgroups' sums added up, in an order that only R and K decide:
// 32 columns per workgroup, eight lanes of four across, 32 rows down.
template <int TY>
__global__ __launch_bounds__(256) void k_norm_join(const float* __restrict__ part, int blocks, int K, void* dw,
                                                   int fp32) {
  __shared__ v4f s_part[32][8];
  const int across = threadIdx.x & 7, down = threadIdx.x >> 3, c = (int(blockIdx.x) * 8 + across) * 4;
  v4f sum = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < K)
    for (int p = down; p < blocks; p += 32) sum += *reinterpret_cast<const v4f*>(part + long(p) * K + c);
  s_part[down][across] = sum;
  __syncthreads();
  if (down || c >= K) return;
#pragma unroll
  for (int u = 1; u < 32; ++u) sum += s_part[u][across];
  if (fp32) {
    *reinterpret_cast<v4f*>(static_cast<float*>(dw) + c) = sum;
  } else {
    typedef __bf16 b4 __attribute__((ext_vector_type(4)));
    typedef _Float16 h4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(dw) + c) =
        TY == kBf16 ? __builtin_bit_cast(uint2, __builtin_convertvector(sum, b4))
                    : __builtin_bit_cast(uint2, __builtin_convertvector(sum, h4));
  }
}

// One launch, or as many as the rows need.
template <int TY, int FMT, int THREADS, int NC>
hipError_t launch_rows(const NormArgs& all, hipStream_t st) {
  constexpr int kBlock = THREADS < 256 ? 256 : THREADS, kPer = kBlock / THREADS;
  constexpr long kMost = max_blocks(kBlock) * kPer;
  for (long r0 = 0; r0 < all.R; r0 += kMost) {
    NormArgs a = all;
    a.R = int(all.R - r0 < kMost ? all.R - r0 : kMost);
    const long at = r0 * a.K;
    auto skip = [](const void* p, long bytes) { return p ? const_cast<char*>(static_cast<const char*>(p)) + bytes : nullptr; };
    a.x = skip(a.x, at * 2);
    a.res = skip(a.res, at * 2);
    a.y = skip(a.y, at * 2);
    a.sum = skip(a.sum, at * 2);
    if (a.rstd) a.rstd += r0;
    a.codes = skip(a.codes, FMT == kQMx4 ? at / 2 : at);
    a.scales = skip(a.scales, FMT == kQMx4 ? at / 32 : FMT == kQE4M3 ? at / a.group * 4 : r0 * 4);
    hipLaunchKernelGGL((k_norm<TY, FMT, THREADS, NC>), dim3(unsigned((a.R + kPer - 1) / kPer)), dim3(kBlock), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// Lanes and chunks: a wave per row up to 1024 values, a workgroup from there on.  (With the
// residual, us: 16384 rows of 1024 in 64 x 2 26.0, 256 x 1 29.8; 16384 of 4096 in 256 x 2 99.8, 512
// x 1 96.4, 512 x 2 93.7, 1024 x 1 103.5; 4099 of 7168 in 256 x 4 50.2, 512 x 2 41.6, 1024 x 1 41.8; 61
// of 7168 4.8, 3.3, 3.1.)
template <int TY, int FMT>
hipError_t launch_fmt(const NormArgs& a, hipStream_t st) {
  if (a.K <= 512) return launch_rows<TY, FMT, 64, 1>(a, st);
  if (a.K <= 1024) return launch_rows<TY, FMT, 64, 2>(a, st);
  if (a.K <= 2048) return launch_rows<TY, FMT, 256, 1>(a, st);
  if (a.K <= 8192) return launch_rows<TY, FMT, 512, 2>(a, st);
  return launch_rows<TY, FMT, 512, 4>(a, st);
}

template <int TY>
hipError_t launch_ty(const NormArgs& a, hipStream_t st) {
  switch (a.fmt) {
    case kQE4M3: return launch_fmt<TY, kQE4M3>(a, st);
    case kQI8: return launch_fmt<TY, kQI8>(a, st);
    case kQMx4: return launch_fmt<TY, kQMx4>(a, st);
    default: return launch_fmt<TY, kQNone>(a, st);
  }
}

template <int TY>
hipError_t launch_grad(const NormGradArgs& a, hipStream_t st) {
  const unsigned grid = unsigned(grad_blocks(a.R, a.K));
  if (grid && (a.dx || a.dw)) {
#define MOE_GRAD(TH, NC) \
  hipLaunchKernelGGL((k_norm_grad<TY, TH, NC>), dim3(grid), dim3(TH < 256 ? 256 : TH), 0, st, a)
    if (a.K <= 512) MOE_GRAD(64, 1);
    else if (a.K <= 1024) MOE_GRAD(64, 2);
    else if (a.K <= 2048) MOE_GRAD(256, 1);
    else if (a.K <= 8192) MOE_GRAD(1024, 1);
    else MOE_GRAD(1024, 2);
#undef MOE_GRAD
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (!a.dw) return hipSuccess;
  hipLaunchKernelGGL((k_norm_join<TY>), dim3(unsigned((a.K + 31) / 32)), dim3(256), 0, st, a.partial, int(grid), a.K,
                     a.dw, a.weight_fp32);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  return a.ty == kBf16 ? launch_ty<kBf16>(a, st) : launch_ty<kFp16>(a, st);
}

size_t norm_grad_bytes(int R, int K) { return size_t(grad_blocks(R, K)) * K * 4; }

hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st) {
  return a.ty == kBf16 ? launch_grad<kBf16>(a, st) : launch_grad<kFp16>(a, st);
}

}  // namespace moe
