// Activations of the linear layers and their derivatives.
//   MLP_ACT_RELU            max(u, 0), f'(0) = 0
//   MLP_ACT_LEAKY_RELU_SQ   (u > 0 ? u : slope u)^2
//   MLP_ACT_GELU            u Phi(u), Phi the normal distribution function
//   MLP_ACT_GELU_TANH       u (1 + tanh z) / 2 = u / (1 + e^(-2z)),
//                           z = sqrt(2 / pi) (u + 0.044715 u^3)
//   MLP_ACT_SILU            u / (1 + e^(-u))
// ACC = true (fp32 layers) uses the CUDA library's functions and its two-ulp
// division (whose quotients read as 0 below about 2^-118).  ACC = false (16-bit
// layers, where the activation's instructions bound the epilogue of short-K
// products) works on two values at a time with the packed fp32 instructions,
// the hardware exponential and reciprocal and, for Phi, a polynomial.
//
// Error of the ACC = false forms, relative to the value itself for f and to the
// sum of magnitudes of its two terms for f' (Phi and u phi; s and u s (1 - s)
// z'): for GELU below 0, 4e-6 + u^2 2^-24; for the logistic ones (4 |z| + 16)
// 2^-23, z the exponential's argument: 5e-5 at most, near 1e-36, and 1e-5 at
// 1e-4.  Above 0, where values are of the order of 1 and u, 3e-7 of 1 + |u|
// (f' of the tanh form up to 5e-6: 1 - s, good to 2^-23, times u z').  Half a
// step of a 16-bit output is 2e-4 (fp16) or more; an fp32 output of a 16-bit
// layer carries these errors.  Values below 2^-120 may read as 0.
#pragma once

#include "f32x2.cuh"

namespace mlp {

// 2^x and 1 / x by the hardware instructions
__device__ __forceinline__ float ex2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// min(|x|, limit); a NaN stays one
__device__ __forceinline__ float abs_upto(float x, float limit) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(x)), "f"(limit));
  return r;
}

// Logistic function of z.
__device__ __forceinline__ F2 sigmoid2(F2 z) {
  const F2 t = mul2(z, f2(-1.4426950408889634f));
  const F2 d = add2(f2(ex2_fast(t.x), ex2_fast(t.y)), f2(1.f));
  return f2(rcp_fast(d.x), rcp_fast(d.y));
}

// Of c = min(|u|, 15): -Phi(-c) and the Gaussian g = e^(-c^2 / 2).  Phi(-c) / g
// falls smoothly from 1/2 to 0.028 at c = 14 (g is 0 from 13.3 on); it is a
// polynomial of degree 7 in t = 1 / (1 + 0.35 c) without a constant term: a
// minimax fit, by linear programming, of its error relative to the ratio,
// weighted so that Phi(-c) is also within 4.2e-8 (2.7e-6 of the ratio, 8.4e-8
// near c = 0), coefficients rounded to fp32.  With the sign turned, u Phi(u) =
// max(u, 0) + c (-Phi(-c)) is one packed instruction.  (Approximation 7.1.26 of
// Abramowitz and Stegun, two terms shorter, bounds the absolute error only: f'
// was 68 % off at u = -6 and f 1 % at -8, in 159 instead of 163 us for the
// backward of 65,536 x 512 -> 1,536 from 8-bit pre-activations.)
__device__ __forceinline__ F2 normal_tail2(F2 c, F2& gauss) {
  const F2 e = mul2(mul2(c, c), f2(-0.72134752044448170f));  // log2(e) / 2
  gauss = f2(ex2_fast(e.x), ex2_fast(e.y));
  const F2 d = fma2(c, f2(0.35f), f2(1.f));
  const F2 t = f2(rcp_fast(d.x), rcp_fast(d.y));
  F2 p = fma2(f2(-0.0449843592941761f), t, f2(0.18593889474868774f));
  p = fma2(p, t, f2(-0.21355803310871124f));
  p = fma2(p, t, f2(-0.0068651409819722176f));
  p = fma2(p, t, f2(-0.1440645009279251f));
  p = fma2(p, t, f2(-0.1366742104291916f));
  p = fma2(p, t, f2(-0.13979268074035645f));
  return mul2(mul2(p, t), gauss);
}

constexpr float kTanhScale = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCubic = 0.044715f;
// Arguments beyond which the bell-shaped parts, Phi(-|u|) and the logistic
// function of -|u| are 0 in fp32: they are evaluated there instead, and the
// factor u that multiplies them is held there from below, so that an infinite u
// gives f and f' their limits rather than 0 times infinity.
constexpr float kGaussEnd = 15.f, kLogisticEnd = 104.f;

// max(u, -limit) of two values; what multiplies it is NaN where u is
__device__ __forceinline__ F2 above2(F2 u, float limit) {
  return f2(fmaxf(u.x, -limit), fmaxf(u.y, -limit));
}

// f(u) of activation ACT for two values.
template <int ACT>
__device__ __forceinline__ F2 act_value2(F2 u, float slope) {
  if constexpr (ACT == MLP_ACT_RELU) {
    return f2(u.x <= 0.f ? 0.f : u.x, u.y <= 0.f ? 0.f : u.y);  // a NaN stays one
  } else if constexpr (ACT == MLP_ACT_LEAKY_RELU_SQ) {
    const F2 s = mul2(u, f2(slope));
    const F2 t = f2(u.x > 0.f ? u.x : s.x, u.y > 0.f ? u.y : s.y);
    return mul2(t, t);
  } else if constexpr (ACT == MLP_ACT_GELU) {
    // u Phi(u) = max(u, 0) - |u| Phi(-|u|)
    const F2 c = f2(abs_upto(u.x, kGaussEnd), abs_upto(u.y, kGaussEnd));
    F2 g;
    const F2 tail = normal_tail2(c, g);
    return fma2(c, tail, f2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
  } else if constexpr (ACT == MLP_ACT_GELU_TANH) {
    const F2 k = fma2(mul2(u, u), f2(kTanhScale * kTanhCubic), f2(kTanhScale));
    return mul2(above2(u, kGaussEnd), sigmoid2(mul2(u, k)));
  } else if constexpr (ACT == MLP_ACT_SILU) {
    return mul2(above2(u, kLogisticEnd), sigmoid2(u));
  } else {
    return u;
  }
}

// f'(u) of two values; f(u) into `value`.
template <int ACT>
__device__ __forceinline__ F2 act_grad2(F2 u, float slope, F2& value) {
  if constexpr (ACT == MLP_ACT_RELU) {
    value = f2(u.x <= 0.f ? 0.f : u.x, u.y <= 0.f ? 0.f : u.y);
    return f2(u.x <= 0.f ? 0.f : 1.f, u.y <= 0.f ? 0.f : 1.f);
  } else if constexpr (ACT == MLP_ACT_LEAKY_RELU_SQ) {
    const F2 s = f2(u.x > 0.f ? 1.f : slope, u.y > 0.f ? 1.f : slope);
    const F2 t = mul2(s, u);
    value = mul2(t, t);
    return mul2(s, add2(t, t));
  } else if constexpr (ACT == MLP_ACT_GELU) {
    const F2 c = f2(abs_upto(u.x, kGaussEnd), abs_upto(u.y, kGaussEnd));
    F2 g;
    const F2 tail = normal_tail2(c, g);
    value = fma2(c, tail, f2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
    // f' = Phi(u) + u phi(u): below 0 that is Phi(-c) - c phi(c), here -d, as it
    // is (no detour over 1, which would leave steps of 2^-24), above it 1 + d
    const F2 d = fma2(mul2(c, f2(0.3989422804014327f)), g, tail);
    const F2 r = add2(d, f2(1.f));
    return f2(u.x < 0.f ? -d.x : r.x, u.y < 0.f ? -d.y : r.y);
  } else if constexpr (ACT == MLP_ACT_GELU_TANH) {
    const F2 c = f2(copysignf(abs_upto(u.x, kGaussEnd), u.x),
                    copysignf(abs_upto(u.y, kGaussEnd), u.y));
    const F2 c2 = mul2(mul2(c, c), f2(kTanhCubic));
    const F2 s = sigmoid2(mul2(mul2(c, f2(kTanhScale)), add2(c2, f2(1.f))));
    value = mul2(above2(u, kGaussEnd), s);
    const F2 w = fma2(c2, f2(3.f * kTanhScale), f2(kTanhScale));
    const F2 b = mul2(mul2(c, s), fma2(s, f2(-1.f), f2(1.f)));
    return fma2(b, w, s);
  } else if constexpr (ACT == MLP_ACT_SILU) {
    const F2 s = sigmoid2(u);  // 0 and 1 beyond the end
    const F2 m = above2(u, kLogisticEnd);
    const F2 c = f2(fminf(m.x, kLogisticEnd), fminf(m.y, kLogisticEnd));
    value = mul2(m, s);
    return fma2(mul2(c, s), fma2(s, f2(-1.f), f2(1.f)), s);
  } else {
    value = u;
    return f2(1.f);
  }
}

// ------------------------------------------------------------ one value

// f(u)
template <bool ACC, int ACT>
__device__ __forceinline__ float act_value_of(float u, float slope) {
  if constexpr (!ACC || ACT <= MLP_ACT_LEAKY_RELU_SQ) {
    return act_value2<ACT>(f2(u), slope).x;
  } else if constexpr (ACT == MLP_ACT_GELU) {
    return fmaxf(u, -kGaussEnd) * 0.5f * erfcf(-0.70710678118654752f * u);
  } else if constexpr (ACT == MLP_ACT_GELU_TANH) {
    return __fdividef(fmaxf(u, -kGaussEnd),
                      1.f + expf(-kTanhScale * fmaf(kTanhCubic * u * u, u, u)));
  } else {
    return __fdividef(fmaxf(u, -kLogisticEnd), 1.f + expf(-u));
  }
}

// f'(u); f(u) into `value`
template <bool ACC, int ACT>
__device__ __forceinline__ float act_grad_of(float u, float slope, float& value) {
  if constexpr (!ACC || ACT <= MLP_ACT_LEAKY_RELU_SQ) {
    F2 v;
    const float d = act_grad2<ACT>(f2(u), slope, v).x;
    value = v.x;
    return d;
  } else if constexpr (ACT == MLP_ACT_GELU) {
    const float c = copysignf(abs_upto(u, kGaussEnd), u);
    const float phi = 0.5f * erfcf(-0.70710678118654752f * c);
    value = fmaxf(u, -kGaussEnd) * phi;
    return fmaf(0.3989422804014327f * c, expf(-0.5f * c * c), phi);
  } else if constexpr (ACT == MLP_ACT_GELU_TANH) {
    const float c = copysignf(abs_upto(u, kGaussEnd), u);
    const float c2 = kTanhCubic * c * c;
    const float s = __fdividef(1.f, 1.f + expf(-kTanhScale * fmaf(c2, c, c)));
    value = fmaxf(u, -kGaussEnd) * s;
    return fmaf(c * s * (1.f - s), kTanhScale * fmaf(3.f, c2, 1.f), s);
  } else {
    const float c = copysignf(abs_upto(u, kLogisticEnd), u);
    const float s = __fdividef(1.f, 1.f + expf(-c));
    value = fmaxf(u, -kLogisticEnd) * s;
    return fmaf(c * s, 1.f - s, s);
  }
}

// Calls f with the activation as a compile-time constant: one branch per call
// instead of one per value.
template <int ACT>
struct ActTag {
  static constexpr int value = ACT;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case MLP_ACT_RELU: f(ActTag<MLP_ACT_RELU>{}); break;
    case MLP_ACT_LEAKY_RELU_SQ: f(ActTag<MLP_ACT_LEAKY_RELU_SQ>{}); break;
    case MLP_ACT_GELU: f(ActTag<MLP_ACT_GELU>{}); break;
    case MLP_ACT_GELU_TANH: f(ActTag<MLP_ACT_GELU_TANH>{}); break;
    case MLP_ACT_SILU: f(ActTag<MLP_ACT_SILU>{}); break;
    default: f(ActTag<MLP_ACT_NONE>{}); break;
  }
}

}  // namespace mlp
