// Pairs of fp32 values and the packed instructions on them: two operations per
// issue slot, each rounded as the single one is.
#pragma once

#include "common.cuh"

namespace mlp {

struct alignas(8) F2 {
  float x, y;
};
__device__ __forceinline__ F2 f2(float a, float b) { return {a, b}; }
__device__ __forceinline__ F2 f2(float a) { return {a, a}; }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  const float2 r = __fmul2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y));
  return {r.x, r.y};
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  const float2 r = __fadd2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y));
  return {r.x, r.y};
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  const float2 r =
      __ffma2_rn(make_float2(a.x, a.y), make_float2(b.x, b.y), make_float2(c.x, c.y));
  return {r.x, r.y};
}

}  // namespace mlp
