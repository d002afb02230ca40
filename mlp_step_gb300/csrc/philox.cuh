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

// What a thread keeps of them.
struct DropKey {
  uint32_t k0, k1, step;
  uint32_t below;  // of 32 bits, whose upper half is a number: dropped up to here
  __device__ __forceinline__ explicit DropKey(const DropArgs& a) : k0(0), k1(0), step(0) {
    below = (a.threshold << 16) - 1u;  // (all ones for a threshold of 2^16)
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

// The random words of the N (4 or 8) values from column c (a multiple of N) of
// `row`: two numbers each, the even column's in the low half.
template <int N>
__device__ __forceinline__ void drop_words(const DropArgs& a, const DropKey& key, uint32_t row,
                                           int c, uint32_t (&w)[N / 2]) {
  uint32_t v[4] = {(uint32_t)c >> 3, row, a.site, key.step};
  philox10(v, key.k0, key.k1);
#pragma unroll
  for (int j = 0; j < N / 2; ++j) w[j] = N == 8 ? v[j] : (c & 4) ? v[2 + j] : v[j];
}

// What is kept of two values times its scale, 0 where dropped (a dropped NaN or
// infinity too).
__device__ __forceinline__ F2 drop2(F2 v, uint32_t word, const DropKey& key, float scale) {
  const F2 s = mul2(v, f2(scale));
  return f2((word << 16) > key.below ? s.x : 0.f, word > key.below ? s.y : 0.f);
}

}  // namespace mlp
