// moe_norm.h -- internal interface between the ABI of the RMS norm
// (moe_norm_api.hip) and its kernels (moe_norm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Forms of the norm's result beside (or in place of) the 16-bit one; the MOE_QFMT_*
// of the ABI, and none.
constexpr int kQE4M3 = 0, kQI8 = 1, kQMx4 = 2, kQNone = 3;

struct NormArgs {
  const void* x;       // [R][K] 16-bit
  const void* res;     // the same, or null
  const void* weight;  // [K] of x's type, or fp32
  void* y;             // [R][K] 16-bit, or null
  void* sum;           // [R][K] 16-bit, or null (always null without res)
  float* rstd;         // [R], or null
  void* codes;         // kQ*
  void* scales;
  int R, K, ty, weight_fp32, fmt, group;
  float eps;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);

struct NormGradArgs {
  const void* dy;      // [R][K]
  const void* dsum;    // [R][K], or null
  const void* sum;     // [R][K]: what was normalised
  const float* rstd;   // [R]
  const void* weight;
  void* dx;            // [R][K], or null
  void* dw;            // [K] of the weight's type, or null
  float* partial;      // norm_grad_bytes() of scratch, or null where that is 0
  int R, K, ty, weight_fp32;
};
size_t norm_grad_bytes(int R, int K);
hipError_t launch_norm_grad(const NormGradArgs& a, hipStream_t st);

}  // namespace moe
