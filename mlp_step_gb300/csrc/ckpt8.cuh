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

// Scale byte of a group from the bits of its largest |x| (whose exponent field
// is 255 for infinity and NaN).
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

// The largest of a running maximum of magnitudes, |x| and |y|; a NaN is kept.
__device__ __forceinline__ float amax_step(float amax, float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(amax), "f"(fabsf(x)), "f"(fabsf(y)));
  return r;
}

// Magnitudes of 127.5 steps and more round to 128 and are held to 127 (a group
// can only hold them when its largest has a mantissa of at least 255/128).
__device__ __forceinline__ bool ckpt8_must_hold(uint32_t amax_bits) {
  return (amax_bits & 0x7fffffu) >= 0x7f0000u;
}
__device__ __forceinline__ float ckpt8_hold(float x, float step) {
  return fminf(fmaxf(x, -127.f * step), 127.f * step);
}

// q of one value (held to 127 steps) as the low byte of the result.  Adding
// 1.5 2^23 rounds x inv_step to a whole number (the product is exact, so the
// fused multiply-add rounds once) and leaves its two's complement in the low
// bits.
__device__ __forceinline__ uint32_t ckpt8_q(float x, float inv_step) {
  return __float_as_uint(fmaf(x, inv_step, 12582912.f));
}

// Four q bytes packed (first value lowest).
__device__ __forceinline__ uint32_t ckpt8_pack4(float a, float b, float c, float d,
                                                float inv_step) {
  const uint32_t lo = __byte_perm(ckpt8_q(a, inv_step), ckpt8_q(b, inv_step), 0x0040);
  const uint32_t hi = __byte_perm(ckpt8_q(c, inv_step), ckpt8_q(d, inv_step), 0x0040);
  return __byte_perm(lo, hi, 0x5410);
}

// A piece of a group: its q bytes, given the largest magnitude of the whole
// group as bits.  Returns the scale byte.
template <int N>
__device__ __forceinline__ uint32_t ckpt8_piece(const float (&v)[N], uint32_t amax_bits,
                                                uint32_t (&w)[N / 4]) {
  const uint32_t b = ckpt8_byte(amax_bits);
  const float inv = ckpt8_inv_step(b);
  if (ckpt8_must_hold(amax_bits)) {  // few groups, and those that are not finite
    const float step = ckpt8_step(b);
#pragma unroll
    for (int k = 0; k < N / 4; ++k)
      w[k] = ckpt8_pack4(ckpt8_hold(v[4 * k], step), ckpt8_hold(v[4 * k + 1], step),
                         ckpt8_hold(v[4 * k + 2], step), ckpt8_hold(v[4 * k + 3], step), inv);
  } else {
#pragma unroll
    for (int k = 0; k < N / 4; ++k)
      w[k] = ckpt8_pack4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3], inv);
  }
  if (b == kCkptNanByte) {
#pragma unroll
    for (int k = 0; k < N / 4; ++k) w[k] = 0u;
  }
  return b;
}

template <int N>
__device__ __forceinline__ uint32_t amax_bits_of(const float (&v)[N]) {
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < N; j += 2) m = amax_step(m, v[j], v[j + 1]);
  return __float_as_uint(m) & 0x7fffffffu;
}

// A whole group held by one thread.
__device__ __forceinline__ uint32_t ckpt8_group(const float (&v)[32], uint32_t (&w)[8]) {
  return ckpt8_piece(v, amax_bits_of(v), w);
}

// The value of byte `i` of a packed word.  Flipping the sign bit makes the
// byte q + 128, which dropped into the low mantissa of 2^23 is an exact float.
constexpr float kCkptBias = 8388736.f;  // 2^23 + 128
__device__ __forceinline__ float ckpt8_biased(uint32_t word_flipped, int i) {
  return __uint_as_float(__byte_perm(word_flipped, 0x4B000000u, 0x7540 + i));
}
__device__ __forceinline__ float ckpt8_value(uint32_t word_flipped, int i, float step) {
  return (ckpt8_biased(word_flipped, i) - kCkptBias) * step;
}
__device__ __forceinline__ uint32_t ckpt8_flip(uint32_t word) { return word ^ 0x80808080u; }

}  // namespace mlp
