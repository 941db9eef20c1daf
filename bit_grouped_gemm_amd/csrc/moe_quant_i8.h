// moe_quant_i8.h -- the int8 quantisation rule on eight values at a time,
// shared by the quantiser and by the products that quantise their own rows.
#pragma once

#include "moe_device.h"
#include "moe_mm.h"

namespace moe {

typedef __bf16 bf8v __attribute__((ext_vector_type(8)));
typedef float f8v __attribute__((ext_vector_type(8)));

typedef int quant_raw8 __attribute__((ext_vector_type(4)));  // eight 16-bit values as they lie in memory

template <int TY>
__device__ __forceinline__ f8v quant_widen8(const quant_raw8& x) {
  if constexpr (TY == kBf16) return __builtin_convertvector(__builtin_bit_cast(bf8v, x), f8v);
  else return __builtin_convertvector(__builtin_bit_cast(h8v, x), f8v);
}

// eight values: x's, or silu(x) * up (GLU)
template <int TY, bool GLU>
__device__ __forceinline__ f8v quant_value8(const quant_raw8& x, const quant_raw8& up) {
  f8v v = quant_widen8<TY>(x);
  if constexpr (GLU) {
    const f8v u = quant_widen8<TY>(up);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = swiglu(v[i], u[i]);
  }
  return v;
}

// the same from column c of a row of K (GLU: of 2 K, gate then up)
template <int TY, bool GLU>
__device__ __forceinline__ f8v quant_value8(const uint16_t* row, int c, int K) {
  const quant_raw8 x = *reinterpret_cast<const quant_raw8*>(row + c);
  return quant_value8<TY, GLU>(x, GLU ? *reinterpret_cast<const quant_raw8*>(row + K + c) : x);
}

// max |v| as bits: they order as the values do, infinities and NaN above all
__device__ __forceinline__ uint32_t quant_top8(const f8v& v) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  return top;
}

// A row's multiplier and scale.  A row that is not finite has codes 0 and the
// scale NaN.
struct QuantScale {
  bool finite;
  float mult, scale;
};
__device__ __forceinline__ QuantScale quant_scale(uint32_t top) {
  QuantScale q;
  q.finite = top < 0x7F800000u;
  q.mult = q.finite ? 127.0f / fmaxf(__uint_as_float(top), 0x1p-64f) : 0.0f;
  q.scale = q.finite ? 1.0f / q.mult : __uint_as_float(0x7FC00000u);
  return q;
}

// eight codes: |v * mult| <= 127 (1 + 2^-23) rounds to at most 127
__device__ __forceinline__ uint2 quant_codes8(const f8v& v, const QuantScale& q) {
  uint32_t o[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    o[h] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = q.finite ? int(__builtin_rintf(v[4 * h + i] * q.mult)) : 0;
      o[h] |= (uint32_t(c) & 0xFFu) << (8 * i);
    }
  }
  return make_uint2(o[0], o[1]);
}

}  // namespace moe
