// moe_mx4.h -- internal interface between the ABI of the row-major MXFP4
// operators (moe_mx4_api.hip) and their kernels (moe_mx4.hip).
#pragma once

#include "moe_mm.h"

namespace moe {

// The product's arguments: p and q hold two e2m1 codes per byte, [rows][K / 2];
// ps, qs, ty and partial are not used.
struct Mx4Args : MmArgs {
  const uint8_t* pe;  // e8m0 per row of p and 32 values of K
  const uint8_t* qe;  // [E][N][K / 32]
};

bool mx4_too_large(const Mx4Args& a);
hipError_t launch_mx4(const Mx4Args& a, hipStream_t st, bool* too_large);

// moe_linear_mx4 of one row as one launch: whether it is, and the launch (a.p:
// the 16-bit rows of type x_ty).
bool linear_mx4_is_one_launch(int R, int K);
hipError_t launch_linear_mx4_one(const Mx4Args& a, int x_ty, int swiglu, hipStream_t st);

// MXFP4 quantisation of rows of `ty` (kBf16 / kFp16): K values per row, or
// SwiGLU of 2 K (gate first).
hipError_t launch_quant_mx4(const void* x, int ty, int swiglu, int R, int K, uint8_t* codes, uint8_t* scales,
                            hipStream_t st);

}  // namespace moe
