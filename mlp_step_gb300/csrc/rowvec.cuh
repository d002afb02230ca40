// 16-byte pieces of matrix rows in fp32 / bf16 / fp16, for the memory-bound
// kernels: a thread's piece is RowVec<T>::N consecutive values, moved as one
// 16-byte access where the row starts on 16 bytes and the piece is whole, and
// value by value at a row's ragged end or for odd row pitches.
#pragma once

#include <type_traits>

#include "f32x2.cuh"

namespace mlp {

template <typename T>
struct RowVec {
  static constexpr int N = 16 / (int)sizeof(T);
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
// one rounding to the nearest, halves to even
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(float v, __half& o) { o = __float2half_rn(v); }

// Two values as one 32-bit word of a 16-bit type, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack_pair(float lo, float hi) {
  if constexpr (std::is_same<T, __half>::value) return pack_f16x2(lo, hi);
  else return pack_bf16x2(lo, hi);
}

// The raw 16 bytes of a piece that starts at p; `n` values of it exist
// (n <= 0: none), the others read as zero.
template <typename T>
__device__ __forceinline__ uint4 load_piece(const T* p, int n, bool vec) {
  constexpr int N = RowVec<T>::N;
  if (vec && n >= N) return *reinterpret_cast<const uint4*>(p);
  union {
    uint4 q;
    T v[N];
  } u;
  u.q = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j < n) u.v[j] = p[j];
  return u.q;
}

template <typename T>
__device__ __forceinline__ void unpack_piece(const uint4& q, float (&v)[RowVec<T>::N]) {
  constexpr int N = RowVec<T>::N;
  const T* h = reinterpret_cast<const T*>(&q);
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = to_f32(h[j]);
}

// The same in pairs.
template <typename T>
__device__ __forceinline__ void unpack_piece(const uint4& q, F2 (&v)[RowVec<T>::N / 2]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(T) == 4) {
    v[0] = f2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[1] = f2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
        v[j] = f2(f.x, f.y);
      } else {
        v[j] = f2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
      }
    }
  }
}

template <typename T>
__device__ __forceinline__ void store_piece(T* p, const float (&v)[RowVec<T>::N], int n, bool vec) {
  constexpr int N = RowVec<T>::N;
  if (vec && n >= N) {
    uint4 q;
    if constexpr (sizeof(T) == 4) {
      q = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                     __float_as_uint(v[3]));
    } else {
      q = make_uint4(pack_pair<T>(v[0], v[1]), pack_pair<T>(v[2], v[3]),
                     pack_pair<T>(v[4], v[5]), pack_pair<T>(v[6], v[7]));
    }
    *reinterpret_cast<uint4*>(p) = q;
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (j < n) from_f32(v[j], p[j]);
}

// FULL: every piece that exists is whole and aligned (rows of whole pieces,
// checked at launch), which leaves only the vector access.
template <bool FULL, typename T>
__device__ __forceinline__ uint4 load_piece_of(const T* p, int n, bool vec) {
  if constexpr (FULL) {
    (void)vec;
    return n > 0 ? *reinterpret_cast<const uint4*>(p) : make_uint4(0, 0, 0, 0);
  } else {
    return load_piece(p, n, vec);
  }
}
template <bool FULL, typename T>
__device__ __forceinline__ void store_piece_of(T* p, const float (&v)[RowVec<T>::N], int n,
                                               bool vec) {
  if constexpr (FULL) {
    if (n > 0) store_piece(p, v, RowVec<T>::N, true);
  } else {
    store_piece(p, v, n, vec);
  }
}

// N consecutive int8 checkpoint values (N 4 or 8) as packed words; the same
// rules, with `vec` meaning the piece starts on N bytes.
template <int N, bool FULL = false>
__device__ __forceinline__ void load_q(const int8_t* p, int n, bool vec, uint32_t (&w)[N / 4]) {
  if (FULL ? n > 0 : vec && n >= N) {
    if constexpr (N == 8) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      w[0] = q.x;
      w[1] = q.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
    return;
  }
#pragma unroll
  for (int k = 0; k < N / 4; ++k) {
    w[k] = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (!FULL && 4 * k + j < n) w[k] |= (uint32_t)(uint8_t)p[4 * k + j] << (8 * j);
  }
}

template <int N, bool FULL = false>
__device__ __forceinline__ void store_q(int8_t* p, int n, bool vec, const uint32_t (&w)[N / 4]) {
  if (FULL ? n > 0 : vec && n >= N) {
    if constexpr (N == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(p) = w[0];
    return;
  }
#pragma unroll
  for (int j = 0; j < N; ++j)
    if (!FULL && j < n) p[j] = (int8_t)(w[j / 4] >> (8 * (j & 3)));
}

}  // namespace mlp
