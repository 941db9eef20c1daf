// moe_quant_mx4.h -- the MXFP4 rule of the row-major operators: 32 consecutive
// values are four lanes' eight, their scale is X = 2^(floor(log2 max |v|) - 2)
// (clamped to the e8m0 range) and the codes are e2m1(v / X).
#pragma once

#include "moe_quant_i8.h"

namespace moe {

constexpr uint32_t kMxNaN = 255;  // e8m0's NaN

// The greatest of four (16) neighbouring lanes' values, in each of them; every lane of
// the wave is active.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ uint32_t group_top_dpp(uint32_t v, int lanes) {
  v = max(v, dpp_u32<0xB1>(v));  // quad_perm [1, 0, 3, 2]
  v = max(v, dpp_u32<0x4E>(v));  // quad_perm [2, 3, 0, 1]
  if (lanes > 4) {
    v = max(v, dpp_u32<0x141>(v));  // row_half_mirror
    v = max(v, dpp_u32<0x140>(v));  // row_mirror
  }
  return v;
}

// The e8m0 byte of a block whose greatest |v| has the bits `top`.
__device__ __forceinline__ uint32_t mx4_scale(uint32_t top) {
  return top < 0x7F800000u ? mx_scale_code(__uint_as_float(top)) : kMxNaN;
}

// Eight codes, the first value's in the lowest four bits; a block that is not
// finite has codes 0.  v / X is exact, and the conversion rounds to nearest even and
// saturates at 6.
__device__ __forceinline__ uint32_t mx4_codes8(const f8v& v, uint32_t scale) {
  if (scale == kMxNaN) return 0;
  const float inv = mx_inv_scale(scale);
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0] * inv, v[1] * inv, 1.0f, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2] * inv, v[3] * inv, 1.0f, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4] * inv, v[5] * inv, 1.0f, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6] * inv, v[7] * inv, 1.0f, 3);
}

}  // namespace moe
