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

// Stochastic rounding of one value x to its code with one random byte r: up
// when the fraction between the two neighbours, times 256, is above r + 0.5.
// From magnitude 1 on, the codes follow the upper bits of an fp32 number: bit
// 22 counts them.  Below 1 they are 1/2 apart; (a + 1) / 2 lies in [1/2, 1),
// where bit 22 counts halves of a, and is above a exactly there, so the larger
// of the two continues the count downwards (code 0 at 1/2).  The magnitude's
// bits plus 2^22 - 1 - (r + 0.5) 2^14 carry into bit 22 exactly when the
// fraction is above the threshold.  (a + 1) / 2 is exact for 16-bit types
// wherever a is above the smallest threshold, 2^-10; for fp32 a is rounded up
// to a multiple of 2^-23 instead, which keeps "above the threshold".
//
// Everything is shifted up by two bits, so that the code is the top byte and
// the random byte a byte too: mx_threshold puts ~r (byte i of rn), the constant
// and minus 1/2's code together in one permutation (10 instructions a value in
// all, 16 without these two steps: both operands of 2048 x 11008 bf16 43 -> 33
// us).
__device__ __forceinline__ uint32_t mx_threshold(uint32_t rn, int i) {
  return __builtin_amdgcn_perm(rn, 0x04007ffcu, 0x03040100u + ((uint32_t)i << 16));
}
template <int DT>
__device__ __forceinline__ uint32_t mx_stochastic(float x, float inv, uint32_t threshold) {
  const float a = fabsf(x) * inv;
  uint32_t bits;
  if (DT == kF32)
    bits = a < 1.f ? 0x3f000000u + (uint32_t)ceilf(a * 0x1p23f) : __float_as_uint(a);
  else
    bits = __float_as_uint(fmaxf(a, fmaf(a, 0.5f, 0.5f)));
  return (bits << 2) + threshold;
}

// Byte B of four words.
template <int B>
__device__ __forceinline__ uint32_t gather_bytes(uint32_t w0, uint32_t w1, uint32_t w2, uint32_t w3) {
  return __builtin_amdgcn_perm(w1, w0, 0x0c0c0400u + B * 0x101u) |
         __builtin_amdgcn_perm(w3, w2, 0x04000c0cu + B * 0x01010000u);
}

// Eight codes (the top bytes of m) and signs (bit 7 of byte E of the words e
// and of byte O of the words o, for the even and the odd values) to a word.
template <int E, int O>
__device__ __forceinline__ uint32_t mx_pack8(const uint32_t (&m)[8], uint32_t e0, uint32_t e1, uint32_t e2, uint32_t e3,
                                             uint32_t o0, uint32_t o1, uint32_t o2, uint32_t o3) {
  const uint32_t even = gather_bytes<3>(m[0], m[2], m[4], m[6]), odd = gather_bytes<3>(m[1], m[3], m[5], m[7]);
  const uint32_t se = gather_bytes<E>(e0, e1, e2, e3) & 0x80808080u;
  const uint32_t so = gather_bytes<O>(o0, o1, o2, o3) & 0x80808080u;
  return even | odd << 4 | se >> 4 | so;
}

// rn: the complements of the eight random bytes.
template <int DT>
__device__ __forceinline__ uint32_t mx_stochastic8(const uint32_t* w, uint32_t byte, const uint32_t* rn) {
  const float inv = byte == 255u ? 0.f : mx_inv_scale(byte);
  uint32_t m[8], q;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = DT == kF32 ? __uint_as_float(w[i]) : Elem<DT>::up((uint16_t)(w[i / 2] >> (i & 1) * 16));
    m[i] = mx_stochastic<DT>(x, inv, mx_threshold(rn[i / 4], i & 3));
  }
  if constexpr (DT == kF32)
    q = mx_pack8<3, 3>(m, w[0], w[2], w[4], w[6], w[1], w[3], w[5], w[7]);
  else
    q = mx_pack8<1, 3>(m, w[0], w[1], w[2], w[3], w[0], w[1], w[2], w[3]);
  return byte == 255u ? 0u : q;
}

// The same for eight words that hold one value each, the half H of a 16-bit
// type's, with a random byte's complement in byte H of rn.
template <int DT, int H>
__device__ __forceinline__ uint32_t mx_stochastic8_column(const uint32_t* w, uint32_t byte, const uint16_t* rn) {
  const float inv = byte == 255u ? 0.f : mx_inv_scale(byte);
  uint32_t m[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = DT == kF32 ? __uint_as_float(w[i]) : Elem<DT>::up((uint16_t)(w[i] >> 16 * H));
    m[i] = mx_stochastic<DT>(x, inv, mx_threshold(rn[i], H));
  }
  constexpr int B = DT == kF32 || H ? 3 : 1;
  const uint32_t q = mx_pack8<B, B>(m, w[0], w[2], w[4], w[6], w[1], w[3], w[5], w[7]);
  return byte == 255u ? 0u : q;
}

// Eight values of DT's words to codes; rn: the complements of their eight
// random bytes.
template <int DT, bool RAND>
__device__ __forceinline__ uint32_t mx_encode8(const uint32_t* w, uint32_t byte, const uint32_t* rn) {
  if constexpr (RAND)
    return mx_stochastic8<DT>(w, byte, rn);
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
