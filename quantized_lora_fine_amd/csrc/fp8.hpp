// Device helpers of the 8-bit floating-point kernels (OCP e4m3 and e5m2).
#pragma once

#include "common.hpp"

namespace nf4k {

constexpr float kFp8Floor = 0x1p-100f;  // the least magnitude a scale is made for

template <bool E5M2>
constexpr float fp8_max() { return E5M2 ? 57344.f : 448.f; }

// Four values to four codes, each rounded to nearest even.  |x| exceeds the
// format's largest value by less than half a step, so nothing overflows; a NaN
// becomes a NaN code.
template <bool E5M2>
__device__ __forceinline__ uint32_t pack_fp8x4(float a, float b, float c, float d) {
  int v = 0;
  if constexpr (E5M2) {
    v = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, v, false);
    v = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, v, true);
  } else {
    v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, v, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
  }
  return (uint32_t)v;
}

// The four codes of a word as fp32 (exact).
template <bool E5M2>
__device__ __forceinline__ void unpack_fp8x4(uint32_t w, float (&v)[4]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  f32x2 lo, hi;
  if constexpr (E5M2) {
    lo = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, false);
    hi = __builtin_amdgcn_cvt_pk_f32_bf8((int)w, true);
  } else {
    lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
    hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  }
  v[0] = lo.x;
  v[1] = lo.y;
  v[2] = hi.x;
  v[3] = hi.y;
}

// Largest of x over the 16 lanes of a DPP row; every lane gets it.  fmaxf takes
// the number where the other operand is a NaN.
__device__ __forceinline__ float row16_max(float x) {
  auto dpp = [](float v, auto ctrl) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF,
                                                              0xF, true));
  };
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0xB1>{}));   // quad_perm [1,0,3,2]
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x4E>{}));   // quad_perm [2,3,0,1]
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x141>{}));  // row_half_mirror
  x = fmaxf(x, dpp(x, std::integral_constant<int, 0x140>{}));  // row_mirror
  return x;
}

// Scale and multiplier of a block whose largest magnitude is amax: codes are
// rne8(fl32(x * mul)) and stand for code * scale.  Both quotients are IEEE
// divisions, and the multiplier is the reciprocal's product with F, which is
// what an array library computes for `F / amax` with a plain number F: such a
// program gets the same codes.  (F / amax rounded once instead differs in the
// last bit for a part of the blocks, and a code in a million falls on the other
// side of a tie.)
template <bool E5M2>
__device__ __forceinline__ void fp8_scale(float amax, float& scale, float& mul) {
  const float m = fmaxf(amax, kFp8Floor);
  scale = m / fp8_max<E5M2>();
  mul = fp8_max<E5M2>() * (1.f / m);
}

__device__ __forceinline__ float abs_max4(float a, float b, float c, float d) {
  return fmaxf(fmaxf(fabsf(a), fabsf(b)), fmaxf(fabsf(c), fabsf(d)));
}

}  // namespace nf4k
