// Device helpers of the microscaled 4-bit format (gfx950).
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "psgd_mx.h"

namespace psgd {

template <int DT>
struct Elem;
template <>
struct Elem<kF32> {
  using type = float;
  static __device__ __forceinline__ float up(float v) { return v; }
  static __device__ __forceinline__ float down(float v) { return v; }
};
template <>
struct Elem<kBF16> {
  using type = uint16_t;
  static __device__ __forceinline__ float up(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
  static __device__ __forceinline__ uint16_t down(float v) {  // nearest, ties to even; a NaN stays a NaN
    const __hip_bfloat16 b = __float2bfloat16(v);
    return __builtin_bit_cast(uint16_t, b);
  }
  static __device__ __forceinline__ uint32_t down2(float v, float w) {  // v in the low half
    typedef float v2f __attribute__((ext_vector_type(2)));
    typedef __bf16 v2b __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((v2f{v, w}), v2b));
  }
};
template <>
struct Elem<kF16> {
  using type = uint16_t;
  static __device__ __forceinline__ float up(uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ __forceinline__ uint16_t down(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
  static __device__ __forceinline__ uint32_t down2(float v, float w) { return down(v) | (uint32_t)down(w) << 16; }
};

// Scale byte of a block whose largest magnitude has the bit pattern `amax`
// (sign bit clear): k + 127 for the smallest k >= -127 with amax <= 6 * 2^k.
// 6 = 1.5 * 2^2, so k is amax's exponent less 2, and one more when its
// fraction is above 1.5: adding 0x3fffff carries into the exponent exactly
// then.  255 (NaN) for a block that holds an infinity or a NaN.
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int e = (int)((amax + 0x3fffffu) >> 23) - 2;
  return (uint32_t)max(e, 0);
}

// 2^-k of a scale byte: 2^(127 - byte), a normal number for every byte up to
// 253 (the largest that a finite block gets).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Eight fp32 values, already times 2^-k (magnitudes at most 6), to eight
// codes, nearest with ties to the even code: the hardware's conversion.
__device__ __forceinline__ uint32_t mx_encode8(const float* v) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], 1.0f, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], 1.0f, 3);
  return r;
}
__device__ __forceinline__ uint32_t mx_encode4(const float* v) {
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], 1.0f, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], 1.0f, 1);
  return r & 0xffffu;
}

// Stochastic rounding of a value already times 2^-k to the format's grid with
// one random byte: up when the fraction between the two neighbours, times
// 256, is above r + 0.5.  Every step is exact in fp32 (the grid's steps are
// powers of two), so the result depends on x and r alone.
__device__ __forceinline__ float mx_stochastic(float x, uint32_t r) {
  const float a = fabsf(x);
  const float step = a < 2.f ? 0.5f : a < 4.f ? 1.f : 2.f;
  const float inv = a < 2.f ? 2.f : a < 4.f ? 1.f : 0.5f;
  const float t = a * inv;
  const float low = floorf(t);
  const float up = (t - low) * 256.f > (float)r + 0.5f ? 1.f : 0.f;
  return copysignf((low + up) * step, x);
}

// Two values of byte `SEL` of a code word, times 2^(byte - 127).
template <int SEL>
__device__ __forceinline__ float2 mx_decode2(uint32_t codes, int k) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, SEL);
  return make_float2(ldexpf(v[0], k), ldexpf(v[1], k));
}

}  // namespace psgd
