// moe_quant_i8.hip -- per-token int8 quantisation of 16-bit rows, optionally
// of their SwiGLU.
//
// One pass over the data: a row's values stay in registers between the
// maximum and the rounding (rows of up to 16384 values; longer ones are read
// again, from L2 as a rule).  Bound by HBM: 2 (SwiGLU: 4) bytes in and one out
// per value.
#include "moe_device.h"
#include "moe_mm.h"

namespace moe {
namespace {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f8v __attribute__((ext_vector_type(8)));

template <int TY>
__device__ __forceinline__ f8v load8(const uint16_t* p) {
  if constexpr (TY == kBf16) return __builtin_convertvector(*reinterpret_cast<const bf8v*>(p), f8v);
  else return __builtin_convertvector(*reinterpret_cast<const h8v*>(p), f8v);
}

// the eight values from column c of a row of K (or 2 K: gate, then up)
template <int TY, bool GLU>
__device__ __forceinline__ f8v value8(const uint16_t* row, int c, int K) {
  f8v v = load8<TY>(row + c);
  if constexpr (GLU) {
    const f8v u = load8<TY>(row + K + c);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = swiglu(v[i], u[i]);
  }
  return v;
}

// THREADS lanes per row (64: four rows per workgroup; 256: one).  NC: chunks
// of 8 values a lane keeps; 0: rows longer than the registers hold.
template <int TY, bool GLU, int THREADS, int NC>
__global__ __launch_bounds__(256) void k_quant_i8(const uint16_t* __restrict__ x, int R, int K,
                                                  int8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t s_max[4];
  const int tid = threadIdx.x % THREADS;
  const long row = long(blockIdx.x) * (256 / THREADS) + threadIdx.x / THREADS;
  const uint16_t* xr = x + row * (GLU ? 2L * K : K);
  constexpr int kKeep = NC > 0 ? NC : 1;
  f8v keep[kKeep];
  // |v| as bits: they order as the values do, infinities and NaN above all
  uint32_t top = 0;
  auto take = [&](const f8v& v) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  };
  if (row < R) {
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (i * THREADS + tid) * 8;
        if (c < K) {
          keep[i] = value8<TY, GLU>(xr, c, K);
          take(keep[i]);
        }
      }
    } else {
      for (int c = tid * 8; c < K; c += THREADS * 8) take(value8<TY, GLU>(xr, c, K));
    }
  }
  for (int d = 1; d < 64; d <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, 64)));
  if constexpr (THREADS == 256) {
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  }
  if (row >= R) return;
  const bool finite = top < 0x7F800000u;
  const float mult = finite ? 127.0f / fmaxf(__uint_as_float(top), 0x1p-64f) : 0.0f;
  if (tid == 0) scales[row] = finite ? 1.0f / mult : __uint_as_float(0x7FC00000u);
  auto put = [&](int c, const f8v& v) __attribute__((always_inline)) {
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      o[h] = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        // |v * mult| <= 127 (1 + 2^-23): rounds to at most 127
        const int q = finite ? int(__builtin_rintf(v[4 * h + i] * mult)) : 0;
        o[h] |= (uint32_t(q) & 0xFFu) << (8 * i);
      }
    }
    *reinterpret_cast<uint2*>(codes + row * K + c) = make_uint2(o[0], o[1]);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      if (c < K) put(c, keep[i]);
    }
  } else {
    for (int c = tid * 8; c < K; c += THREADS * 8) put(c, value8<TY, GLU>(xr, c, K));
  }
}

template <int TY, bool GLU>
hipError_t launch_ty(const uint16_t* x, int R, int K, int8_t* codes, float* scales, hipStream_t st) {
#define MOE_QUANT(TH, NC)                                                                                       \
  hipLaunchKernelGGL((k_quant_i8<TY, GLU, TH, NC>), dim3((long(R) * TH + 255) / 256), dim3(256), 0, st, x, R, K, \
                     codes, scales)
  // a wave per row while its lanes hold the row in two chunks each
  if (K <= 512) MOE_QUANT(64, 1);
  else if (K <= 1024) MOE_QUANT(64, 2);
  else if (K <= 2048) MOE_QUANT(256, 1);
  else if (K <= 4096) MOE_QUANT(256, 2);
  else if (K <= 8192) MOE_QUANT(256, 4);
  else if (K <= 16384) MOE_QUANT(256, 8);
  else MOE_QUANT(256, 0);
#undef MOE_QUANT
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_i8(const void* x, int ty, int swiglu, int R, int K, int8_t* codes, float* scales,
                           hipStream_t st) {
  if (R == 0) return hipSuccess;
  const uint16_t* xs = static_cast<const uint16_t*>(x);
  if (ty == kBf16)
    return swiglu ? launch_ty<kBf16, true>(xs, R, K, codes, scales, st)
                  : launch_ty<kBf16, false>(xs, R, K, codes, scales, st);
  return swiglu ? launch_ty<kFp16, true>(xs, R, K, codes, scales, st)
                : launch_ty<kFp16, false>(xs, R, K, codes, scales, st);
}

}  // namespace moe
