// moe_quant_i8.hip -- per-token int8 quantisation of 16-bit rows, optionally
// of their SwiGLU.
//
// One pass over the data: a row's values stay in registers between the
// maximum and the rounding (rows of up to 16384 values; longer ones are read
// again, from L2 as a rule).  Bound by HBM: 2 (SwiGLU: 4) bytes in and one out
// per value; 32768 rows of 7168: 127 us, 5.5 TB/s; SwiGLU of 32768 rows of 2048: 77
// us, 4.4 TB/s.
#include "moe_quant_i8.h"

namespace moe {
namespace {

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
  uint32_t top = 0;
  if (row < R) {
    if constexpr (NC > 0) {
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (i * THREADS + tid) * 8;
        if (c < K) {
          keep[i] = quant_value8<TY, GLU>(xr, c, K);
          top = max(top, quant_top8(keep[i]));
        }
      }
    } else {
      for (int c = tid * 8; c < K; c += THREADS * 8) top = max(top, quant_top8(quant_value8<TY, GLU>(xr, c, K)));
    }
  }
  for (int d = 1; d < 64; d <<= 1) top = max(top, uint32_t(__shfl_xor(int(top), d, 64)));
  if constexpr (THREADS == 256) {
    if ((threadIdx.x & 63) == 0) s_max[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  }
  if (row >= R) return;
  const QuantScale q = quant_scale(top);
  if (tid == 0) scales[row] = q.scale;
  auto put = [&](int c, const f8v& v) __attribute__((always_inline)) {
    *reinterpret_cast<uint2*>(codes + row * K + c) = quant_codes8(v, q);
  };
  if constexpr (NC > 0) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (i * THREADS + tid) * 8;
      if (c < K) put(c, keep[i]);
    }
  } else {
    for (int c = tid * 8; c < K; c += THREADS * 8) put(c, quant_value8<TY, GLU>(xr, c, K));
  }
}

// One launch, or as many as the rows need: THREADS = 64 passes a launch's limit
// at 2^26 rows (2 GB of x at K = 16), THREADS = 256 at 2^24.
template <int TY, bool GLU, int THREADS, int NC>
hipError_t launch_rows(const uint16_t* x, int R, int K, int8_t* codes, float* scales, hipStream_t st) {
  constexpr int kPer = 256 / THREADS;  // rows of a workgroup
  constexpr long kMost = max_blocks(256) * kPer;
  for (long r0 = 0; r0 < R; r0 += kMost) {
    const long n = R - r0 < kMost ? R - r0 : kMost;
    hipLaunchKernelGGL((k_quant_i8<TY, GLU, THREADS, NC>), dim3(unsigned((n + kPer - 1) / kPer)), dim3(256), 0, st,
                       x + r0 * (GLU ? 2L * K : K), int(n), K, codes + r0 * K, scales + r0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <int TY, bool GLU>
hipError_t launch_ty(const uint16_t* x, int R, int K, int8_t* codes, float* scales, hipStream_t st) {
#define MOE_QUANT(TH, NC) return launch_rows<TY, GLU, TH, NC>(x, R, K, codes, scales, st)
  // a wave per row up to 1024 values, a workgroup from there on (32768 rows:
  // K = 1024 17.4 us against 25.5, K = 2048 33.0 against 33.1, K = 4096 78
  // against 69; 488 rows of 1536, SwiGLU: 4.4 against 3.5)
  if (K <= 512) MOE_QUANT(64, 1);
  else if (K <= 1024) MOE_QUANT(64, 2);
  else if (K <= 2048) MOE_QUANT(256, 1);
  else if (K <= 4096) MOE_QUANT(256, 2);
  else if (K <= 8192) MOE_QUANT(256, 4);
  else if (K <= 16384) MOE_QUANT(256, 8);
  else MOE_QUANT(256, 0);
#undef MOE_QUANT
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
