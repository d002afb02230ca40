// The 8-bit activation checkpoint format (include/mlp_step.h): 32 consecutive
// values of a row share one scale byte b, and a stored int8 q stands for
// q 2^(b - 133).  b is the fp32 exponent field of the group's largest
// magnitude (so |x| 2^(133 - b) < 128), at least 7 (steps of 2^-126 and up
// keep both powers of two normal fp32 numbers), and 255 for a group that held
// an infinity or NaN, which reads back as NaN.  Power-of-two steps make the
// scaling exact in fp32: the one rounding is to the nearest whole q (halves to
// even), and magnitudes that round to 128 are held to 127.
#pragma once

#include "common.cuh"

namespace mlp {

constexpr int kCkptGroup = 32;
constexpr uint32_t kCkptMinByte = 7, kCkptNanByte = 255;

// Scale byte of a group from the largest |x| of it as fp32 bits (compared as
// whole numbers, in which NaN and infinity are the largest).
__device__ __forceinline__ uint32_t ckpt8_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e < kCkptMinByte ? kCkptMinByte : e;
}

// 2^(133 - b)
__device__ __forceinline__ float ckpt8_inv_step(uint32_t b) {
  return __uint_as_float((260u - b) << 23);
}

// 2^(b - 133), or NaN for the byte of a group that was not finite
__device__ __forceinline__ float ckpt8_step(uint32_t b) {
  if (b < kCkptMinByte) b = kCkptMinByte;
  return __uint_as_float(b == kCkptNanByte ? 0x7fffffffu : (b - 6u) << 23);
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// q of one value as the low byte of the result.  Adding 1.5 2^23 rounds
// x inv_step to a whole number (the product is exact, so the fused
// multiply-add rounds once) and leaves its two's complement in the low bits;
// the clamp is on the sum, where whole steps are exact.
__device__ __forceinline__ uint32_t ckpt8_q(float x, float inv_step) {
  constexpr float kMagic = 12582912.f;
  const float t = fmaf(x, inv_step, kMagic);
  return __float_as_uint(fminf(fmaxf(t, kMagic - 127.f), kMagic + 127.f));
}

// Four q bytes packed (first value lowest).
__device__ __forceinline__ uint32_t ckpt8_pack4(float a, float b, float c, float d,
                                                float inv_step) {
  const uint32_t lo = __byte_perm(ckpt8_q(a, inv_step), ckpt8_q(b, inv_step), 0x0040);
  const uint32_t hi = __byte_perm(ckpt8_q(c, inv_step), ckpt8_q(d, inv_step), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// The value of byte `i` of a packed word.  Flipping the sign bit makes the
// byte q + 128, which dropped into the low mantissa of 2^23 is an exact float.
__device__ __forceinline__ float ckpt8_value(uint32_t word_flipped, int i, float step) {
  const uint32_t f = __byte_perm(word_flipped, 0x4B000000u, 0x7540 + i);
  return (__uint_as_float(f) - 8388736.f) * step;
}
__device__ __forceinline__ uint32_t ckpt8_flip(uint32_t word) { return word ^ 0x80808080u; }

}  // namespace mlp
