// Device pieces of the microscaled formats: 32 columns share a scale 2^(s - 127),
// s a byte (255: NaN); their elements are e4m3 (a byte) or e2m1 (half a byte).
#pragma once

#include "layer_device.hpp"
#include "layer_launch.hpp"

namespace flce {

// The largest of a value over the four lanes that hold a scale's 32 columns.
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));   // lanes 1 0 3 2
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));   // lanes 2 3 0 1
}

// The scale byte of a block whose largest magnitude has these bits:
// floor(log2(largest)) less the format's largest exponent, biased, not below 0.
// Infinity and NaN, whose bits are the largest, give 255.  Magnitudes are compared
// as bits, so a NaN is never lost.
template <int FMT> __device__ __forceinline__ uint32_t mx_scale(uint32_t bits) {
  constexpr int emax = FMT == kMxE4M3 ? 8 : 2;
  const int e = (int)(bits >> 23) - emax;
  return bits >= 0x7f800000u ? 255u : (uint32_t)(e < 0 ? 0 : e);
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// 2^(s - 127) for s < 255.  s = 0 is a subnormal float.
__device__ __forceinline__ float mx_scale_value(uint32_t s) { return __uint_as_float(s ? s << 23 : 0x400000u); }

// Eight elements under scale byte s, each v 2^(127 - s) rounded to nearest, ties
// to even, and held to the format's largest (448; the e2m1 conversion saturates
// by itself).  The conversions take the scale's exponent bits; a subnormal scale
// would be read as 0, so for s = 0 the values are scaled up by 2^32 first (they are
// under 2^-118) and the scale with them, both exact.
template <int FMT> __device__ __forceinline__ void mx_encode(const float (&x)[8], uint32_t s, uint32_t (&code)[2]) {
  float v[8];
  const bool low = s == 0;
  const float scale = low ? __uint_as_float(32u << 23) : __uint_as_float(s << 23);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = low ? x[e] * 4294967296.f : x[e];
  if constexpr (FMT == kMxE4M3) {
    const float lim = 448.f * scale;
    typedef short s16x2 __attribute__((ext_vector_type(2)));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      s16x2 r = {0, 0};
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * h + e] = __builtin_amdgcn_fmed3f(v[4 * h + e], -lim, lim);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * h], v[4 * h + 1], scale, false);
      r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, v[4 * h + 2], v[4 * h + 3], scale, true);
      code[h] = s == 255 ? 0u : __builtin_bit_cast(uint32_t, r);
    }
  } else {
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], scale, 3);
    code[0] = s == 255 ? 0u : r;
    code[1] = 0u;
  }
}

// Eight elements' values: codes lo and hi (e2m1: lo alone) times 2^(s - 127); a block
// of scale 255 is NaN.  fp32's subnormals hold what is left of the smallest.
template <int FMT> __device__ __forceinline__ void mx_decode8(uint32_t lo, uint32_t hi, uint32_t s, float (&v)[8]) {
  const float scale = s == 255 ? __uint_as_float(0x7fc00000u) : mx_scale_value(s);
  f32x2 p[4];
  if constexpr (FMT == kMxE4M3) {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 1.f, false);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(lo, 1.f, true);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 1.f, false);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(hi, 1.f, true);
  } else {
    p[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.f, 0);
    p[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.f, 1);
    p[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.f, 2);
    p[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo, 1.f, 3);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    v[2 * k] = p[k][0] * scale;
    v[2 * k + 1] = p[k][1] * scale;
  }
}

// Eight float32 values of a row's columns col .. col + 7 (in four adjacent lanes, 32
// columns) to their place among its codes and scales.
template <int FMT>
__device__ __forceinline__ void mx_store8(uint8_t* codes, uint8_t* scales, int64_t row, int Cp, int col, const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, abs_bits(v[e]));
  const uint32_t s = mx_scale<FMT>(quad_max(top));
  uint32_t code[2];
  mx_encode<FMT>(v, s, code);
  if (col >= Cp) return;
  if constexpr (FMT == kMxE4M3) *(u32x2*)(codes + row * Cp + col) = u32x2{code[0], code[1]};
  else *(uint32_t*)(codes + row * (Cp / 2) + col / 2) = code[0];
  if ((col & 31) == 0) scales[row * (Cp / kMxBlock) + col / kMxBlock] = (uint8_t)s;
}

}  // namespace flce
