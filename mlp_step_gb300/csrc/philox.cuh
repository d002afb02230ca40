// Dropout's random numbers: Philox4x32-10, the counter-based generator of
// Salmon, Moraes, Dror and Shaw ("Parallel random numbers: as easy as 1, 2, 3",
// 2011).  Whether value (row, column) is kept depends on its place alone: the
// counter is (column / 8, row, site, step), the key the seed, and the four
// words are eight 16-bit numbers, low halves first, for eight neighbouring
// columns.  So the mask is never stored: the backward, another tile shape or
// another type computes the same one.
#pragma once

#include "f32x2.cuh"

namespace mlp {

struct DropArgs {
  const unsigned long long* rng;  // device: seed, step (its low 32 bits count)
  uint32_t site;
  uint32_t threshold;  // numbers below it drop: p in steps of 2^-16; 0: no dropout
  float scale;         // of what is kept: 2^16 / (2^16 - threshold), 0 where nothing is
};

struct DropKey {
  uint32_t k0, k1, step;
  __device__ __forceinline__ explicit DropKey(const DropArgs& a) : k0(0), k1(0), step(0) {
    if (a.threshold) {
      const unsigned long long seed = a.rng[0];
      k0 = (uint32_t)seed;
      k1 = (uint32_t)(seed >> 32);
      step = (uint32_t)a.rng[1];
    }
  }
};

__device__ __forceinline__ void philox10(uint32_t (&c)[4], uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)c[0] * 0xD2511F53u, b = (uint64_t)c[2] * 0xCD9E8D57u;
    const uint32_t n0 = (uint32_t)(b >> 32) ^ c[1] ^ (k0 + i * 0x9E3779B9u);
    const uint32_t n2 = (uint32_t)(a >> 32) ^ c[3] ^ (k1 + i * 0xBB67AE85u);
    c[0] = n0;
    c[1] = (uint32_t)b;
    c[2] = n2;
    c[3] = (uint32_t)a;
  }
}

// Bit j: value j of the N (4 or 8) from column c (a multiple of N) of `row` is kept.
template <int N>
__device__ __forceinline__ uint32_t drop_bits(const DropArgs& a, const DropKey& key, uint32_t row,
                                              int c) {
  uint32_t w[4] = {(uint32_t)c >> 3, row, a.site, key.step};
  philox10(w, key.k0, key.k1);
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < N / 2; ++j) {
    const uint32_t v = N == 8 ? w[j] : (c & 4) ? w[2 + j] : w[j];
    bits |= (uint32_t)((v & 0xffffu) >= a.threshold) << (2 * j);
    bits |= (uint32_t)((v >> 16) >= a.threshold) << (2 * j + 1);
  }
  return bits;
}

// What is kept times its scale, 0 where dropped (a dropped NaN or infinity too).
__device__ __forceinline__ F2 drop2(F2 v, uint32_t bits, int j, float scale) {
  const F2 s = mul2(v, f2(scale));
  return f2(bits >> j & 1 ? s.x : 0.f, bits >> (j + 1) & 1 ? s.y : 0.f);
}

}  // namespace mlp
