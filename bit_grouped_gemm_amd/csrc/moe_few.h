// moe_few.h -- internal interface between the ABI of the few-token layer on
// 16-bit row-major weights (moe_few_api.hip) and its kernels (moe_few.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kFewTokens = 64;  // most tokens of a call

struct FewArgs {
  const void* x;         // [T][H]
  const int32_t* ids;    // [T][k]
  const float* weights;  // [T][k]
  const void* w1;        // [E][2 I][H]
  const void* w2;        // [E][H][I]
  void* out;             // [T][H]
  int T, H, I, E, k, ty;
  // workspace
  int32_t* count;        // row tiles, 1 int
  int2* tiles;           // [row tiles]: expert, rows
  int32_t* slots;        // [row tiles][rows of a tile: 8, 16 or 32]
  uint16_t *hi, *lo;     // [T * k][I]: h as the sum of two 16-bit values
  float* partial;        // sums of the second product, where workgroups share columns
};

size_t few_bytes(int T, int H, int I, int E, int k);
void few_carve(FewArgs& a, void* ws);
hipError_t launch_few(const FewArgs& a, hipStream_t st);

}  // namespace moe
