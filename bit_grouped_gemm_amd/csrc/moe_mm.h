// moe_mm.h -- internal interface between the ABI of the row-major products
// (moe_mm_api.hip) and their kernels (moe_mm.hip, moe_quant_i8.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

// Operand types of the products and element types of their outputs
// (MOE_DT_* of the ABI; int8 is internal).
constexpr int kBf16 = 0, kFp16 = 1, kFp32 = 2, kInt8 = 3;

// The three products over ragged groups e of rows r:
//   kFwd    y[r][n]  = sum_k x[r][k]  w[e][n][k]   (reduction K)
//   kDgrad  dx[r][k] = sum_n dy[r][n] w[e][n][k]   (reduction N)
//   kWgrad  dw[e][n][k] = sum_{r in e} dy[r][n] x[r][k]
constexpr int kFwd = 0, kDgrad = 1, kWgrad = 2;

// Workgroups of `threads` that one launch may have: its work items are counted
// in 32 bits, and a count past them wraps, so that most of the grid never runs
// and the call still succeeds.
constexpr long max_blocks(int threads) { return ((1L << 32) - 1) / threads; }
static_assert(max_blocks(256) * 256 < (1L << 32) && (max_blocks(256) + 1) * 256 >= (1L << 32), "limit of a launch");

struct MmArgs {
  const void* p;             // x (kFwd) or dy: the operand whose index is the output's row
  const void* q;             // w, or x (kWgrad): its index is the output's column
  void* out;
  const int32_t* offsets;    // [E + 1]; null: one group of R rows
  const int32_t* row_token;  // int8 only: row of p for each output row, or null
  const float* ps;           // int8 only: scale per row of p
  const float* qs;           // int8 only: scale per [E][N]
  int R, N, K, E, T;
  int ty;                    // operand type
  int out_ty;                // output type
  int clear_rest;            // rows of no group: 1 written as zeros, 0 left alone
  float* partial;            // kWgrad: wgrad_bytes() of scratch, or null where that is 0
  int splits;                // set by launch_mm
};

// Scratch of kWgrad.
size_t wgrad_bytes(const MmArgs& a);
// Whether a product needs more workgroups than a launch has, and its launch
// (*too_large: nothing was enqueued for that reason).
bool mm_too_large(int op, const MmArgs& a);
hipError_t launch_mm(int op, const MmArgs& a, hipStream_t st, bool* too_large);

// moe_linear_i8 of one row as one launch: whether it is, and the launch (a.p:
// the 16-bit rows of type x_ty).
bool linear_is_one_launch(int R, int K);
hipError_t launch_linear_one(const MmArgs& a, int x_ty, int swiglu, hipStream_t st);

// Per-token int8 quantisation of rows of `ty` (kBf16 / kFp16): K values per
// row, or SwiGLU of 2 K (gate first).
hipError_t launch_quant_i8(const void* x, int ty, int swiglu, int R, int K, int8_t* codes, float* scales,
                           hipStream_t st);

}  // namespace moe
