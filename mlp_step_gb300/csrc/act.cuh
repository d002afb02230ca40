// Activations of the linear layers and their derivatives.
//   MLP_ACT_RELU            max(u, 0), f'(0) = 0
//   MLP_ACT_LEAKY_RELU_SQ   (u > 0 ? u : slope u)^2
//   MLP_ACT_GELU            u Phi(u), Phi the normal distribution function
//   MLP_ACT_GELU_TANH       u (1 + tanh z) / 2 = u / (1 + e^(-2z)),
//                           z = sqrt(2 / pi) (u + 0.044715 u^3)
//   MLP_ACT_SILU            u / (1 + e^(-u))
// ACC = true uses the CUDA library functions (fp32 operands); ACC = false the
// hardware exponential and reciprocal (a few 2^-23 relative) and, for Phi,
// the rational approximation 7.1.26 of Abramowitz and Stegun, "Handbook of
// Mathematical Functions" (absolute error 1.5e-7 of erfc): below the rounding
// of 16-bit outputs, and about half the instructions, which bound the
// epilogue of short-K products.
#pragma once

#include "common.cuh"

namespace mlp {

// 2^x by the hardware instruction
__device__ __forceinline__ float exp2f_fast(float x) {
  float r;
  asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <bool ACC>
__device__ __forceinline__ float act_sigmoid(float z) {
  if constexpr (ACC) return 1.f / (1.f + expf(-z));
  else return __fdividef(1.f, 1.f + __expf(-z));
}

// Phi(u), and e^(-u^2 / 2) on the way
template <bool ACC>
__device__ __forceinline__ float act_phi(float u, float& gauss) {
  if constexpr (ACC) {
    gauss = expf(-0.5f * u * u);
    return 0.5f * erfcf(-0.70710678118654752f * u);
  } else {
    gauss = exp2f_fast(-0.72134752044448170f * u * u);  // log2(e) / 2
    const float t = __fdividef(1.f, fmaf(0.23164188612f, fabsf(u), 1.f));  // 0.3275911 / sqrt 2
    // half of a1 .. a5
    float p = fmaf(0.5307027145f, t, -0.7265760135f);
    p = fmaf(p, t, 0.7107068705f);
    p = fmaf(p, t, -0.142248368f);
    p = fmaf(p, t, 0.127414796f);
    const float tail = p * t * gauss;  // Phi(-|u|)
    return u < 0.f ? tail : 1.f - tail;
  }
}

template <bool ACC>
__device__ __forceinline__ float act_value(float u, int act, float slope) {
  switch (act) {
    case MLP_ACT_RELU: return u <= 0.f ? 0.f : u;  // a NaN stays one
    case MLP_ACT_LEAKY_RELU_SQ: {
      const float t = u > 0.f ? u : slope * u;
      return t * t;
    }
    case MLP_ACT_GELU: {
      float g;
      return u * act_phi<ACC>(u, g);
    }
    case MLP_ACT_GELU_TANH:
      return u * act_sigmoid<ACC>(1.5957691216057308f * fmaf(0.044715f * u * u, u, u));
    case MLP_ACT_SILU: return u * act_sigmoid<ACC>(u);
    default: return u;
  }
}

// f'(u); f(u) into `value`.  Arguments of the bell-shaped parts are held to
// where those parts are below the smallest fp32 (|u| = 14 for the Gaussian
// and the cubic, 104 for the logistic), so that an infinite u gives the
// limits 0 and 1 rather than 0 times infinity.
template <bool ACC>
__device__ __forceinline__ float act_grad(float u, int act, float slope, float& value) {
  switch (act) {
    case MLP_ACT_RELU:
      value = u <= 0.f ? 0.f : u;
      return u <= 0.f ? 0.f : 1.f;
    case MLP_ACT_LEAKY_RELU_SQ: {
      const float s = u > 0.f ? 1.f : slope;
      const float t = s * u;
      value = t * t;
      return 2.f * s * t;
    }
    case MLP_ACT_GELU: {
      const float c = fabsf(u) > 14.f ? copysignf(14.f, u) : u;
      float g;
      const float phi = act_phi<ACC>(c, g);
      value = u * phi;
      return fmaf(0.3989422804014327f * c, g, phi);
    }
    case MLP_ACT_GELU_TANH: {
      const float c = fabsf(u) > 14.f ? copysignf(14.f, u) : u;
      const float c2 = 0.044715f * c * c;
      const float s = act_sigmoid<ACC>(1.5957691216057308f * fmaf(c2, c, c));
      value = u * s;
      return fmaf(c * s * (1.f - s), 1.5957691216057308f * fmaf(3.f, c2, 1.f), s);
    }
    case MLP_ACT_SILU: {
      const float c = fabsf(u) > 104.f ? copysignf(104.f, u) : u;
      const float s = act_sigmoid<ACC>(c);
      value = u * s;
      return fmaf(c * s, 1.f - s, s);
    }
    default:
      value = u;
      return 1.f;
  }
}

}  // namespace mlp
