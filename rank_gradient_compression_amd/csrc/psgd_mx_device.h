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

// Runs of values are handled as the words they are loaded in: one fp32 value
// or two 16-bit ones to a word.
template <int DT>
constexpr int kPerWord = 4 / dtype_bytes(DT);

// Largest magnitude of N words, as the bits of an fp32 value (sign clear).
// The bit patterns of every type order like the magnitudes, infinities and
// NaN above all finite values.
__device__ __forceinline__ uint32_t mx_pk_max(uint32_t a, uint32_t b) {
  typedef uint16_t v2s __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(v2s, a), __builtin_bit_cast(v2s, b)));
}
template <int DT>
__device__ __forceinline__ uint32_t mx_max_words(uint32_t m, uint32_t w) {
  return DT == kF32 ? max(m, w & 0x7fffffffu) : mx_pk_max(m, w & 0x7fff7fffu);
}
template <int DT>
__device__ __forceinline__ uint32_t mx_half_max_bits(uint32_t h) {  // of a 16-bit pattern
  return DT == kBF16 ? h << 16 : __float_as_uint(Elem<kF16>::up((uint16_t)h));
}
template <int DT>
__device__ __forceinline__ uint32_t mx_max_bits(uint32_t m) {
  return DT == kF32 ? m : mx_half_max_bits<DT>(max(m & 0xffffu, m >> 16));
}

// Eight values to eight codes of x * 2^-k, nearest with ties to the even code:
// the hardware's conversion, which takes 2^k and the values as they are.
// (Every step is exact but the one rounding; byte 255 gives zero codes.)
template <int DT>
__device__ __forceinline__ uint32_t mx_nearest8(const uint32_t* w, uint32_t byte) {
  typedef __bf16 v2b __attribute__((ext_vector_type(2)));
  typedef _Float16 v2h __attribute__((ext_vector_type(2)));
  const float scale = __uint_as_float(byte << 23);
  uint32_t r = 0;
  if constexpr (DT == kF32) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[0]), __uint_as_float(w[1]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[2]), __uint_as_float(w[3]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[4]), __uint_as_float(w[5]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, __uint_as_float(w[6]), __uint_as_float(w[7]), scale, 3);
  } else if constexpr (DT == kBF16) {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2b, w[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2b, w[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2b, w[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(v2b, w[3]), scale, 3);
  } else {
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, w[0]), scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, w[1]), scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, w[2]), scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(r, __builtin_bit_cast(v2h, w[3]), scale, 3);
  }
  return byte == 255u ? 0u : r;
}

// Stochastic rounding of one value to its code with one random byte r: up when
// the fraction between the two neighbours, times 256, is above r + 0.5.  From
// magnitude 1 on the code's spacing is bit 22 of an fp32 number (one fraction
// bit), below it is 1/2: in either case the magnitude, as an integer whose
// bit 22 counts codes, plus 2^22 - 1 - (r + 0.5) 2^14 carries into bit 22
// exactly when the fraction is above the threshold.  Below 1 the integer is
// a * 2^23: exact for 16-bit types (a value above the smallest threshold, 2^13,
// has its 11 bits or fewer above 1), rounded up for fp32, which keeps "above
// the threshold".  (All values are doubled here, to shift the sign out.)
template <int DT>
__device__ __forceinline__ uint32_t mx_stochastic_code(float x, float inv, uint32_t r) {
  const float t = x * inv, a = fabsf(t);
  const uint32_t big = (__float_as_uint(t) << 1) - (0xFCu << 23);
  const uint32_t small = DT == kF32 ? (uint32_t)ceilf(a * 0x1p23f) << 1 : (uint32_t)(a * 0x1p24f);
  const uint32_t m = (a < 1.f ? small : big) + (2u * (0x3fffffu - 0x2000u) - (r << 15));
  return (m >> 23) | (__float_as_uint(x) >> 28 & 8u);
}
template <int DT>
__device__ __forceinline__ uint32_t mx_stochastic8(const uint32_t* w, uint32_t byte, const uint32_t* rnd) {
  const float inv = byte == 255u ? 0.f : mx_inv_scale(byte);
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = DT == kF32 ? __uint_as_float(w[i]) : Elem<DT>::up((uint16_t)(w[i / 2] >> (i & 1) * 16));
    q |= mx_stochastic_code<DT>(x, inv, rnd[i / 4] >> (i & 3) * 8 & 255u) << 4 * i;
  }
  return byte == 255u ? 0u : q;
}

// Eight values of DT's words to codes; rnd: their eight random bytes.
template <int DT, bool RAND>
__device__ __forceinline__ uint32_t mx_encode8(const uint32_t* w, uint32_t byte, const uint32_t* rnd) {
  if constexpr (RAND)
    return mx_stochastic8<DT>(w, byte, rnd);
  else
    return mx_nearest8<DT>(w, byte);
}

// Workgroup b of `total` to a position in the walk over a matrix's tiles:
// consecutive workgroups go to the eight XCDs in turn, each with an L2 of its
// own, so XCD x takes the x-th eighth of the walk.
__device__ __forceinline__ int xcd_position(int b, int total) {
  const int q = total / 8, rem = total % 8, x = b % 8;
  return x * q + min(x, rem) + b / 8;
}

// Two values of byte `SEL` of a code word, times 2^(byte - 127).
template <int SEL>
__device__ __forceinline__ float2 mx_decode2(uint32_t codes, int k) {
  typedef float v2f __attribute__((ext_vector_type(2)));
  const v2f v = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, SEL);
  return make_float2(ldexpf(v[0], k), ldexpf(v[1], k));
}

}  // namespace psgd
