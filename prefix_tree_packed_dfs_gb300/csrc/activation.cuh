// Activations of the projections and the feed-forward block, and their
// derivatives, in fp32 (include/tpk.h, TPK_ACT_*).
//   silu       z s,  s = 1 / (1 + e^-z)            s (1 + z (1 - s))
//   gelu       z Phi(z)                            Phi(z) + z phi(z)
//   gelu_tanh  z s(k (z + c z^3)), k = 2 sqrt(2 / pi), c = 0.044715
//              (0.5 (1 + tanh t) = s(2 t): no difference of close numbers)
// Phi through erfc(x) ~ (a1 t + .. + a5 t^5) e^{-x^2}, t = 1 / (1 + p x), for
// x >= 0 (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26):
// within 1.5e-7, far inside the results' bf16 rounding, at a third of the
// instructions of the full-precision function, and the derivative shares the
// exponential.
#pragma once
#include "ptx.cuh"
#include "tpk.h"

namespace tpk {

constexpr float kActLog2e = 1.4426950408889634f;

__device__ __forceinline__ float sigmoid_of(float z) { return __fdividef(1.f, 1.f + ptx::ex2(-z * kActLog2e)); }

// (erfc(|z| / sqrt 2), e^{-z^2 / 2})
__device__ __forceinline__ void tail_of(float z, float& q, float& e) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  e = ptx::ex2(z * z * (-0.5f * kActLog2e));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  q = p * t * e;
}

__device__ __forceinline__ float tanh_arg(float z) {
  constexpr float k = 1.5957691216057308f;   // 2 sqrt(2 / pi)
  return z * fmaf(0.044715f * k, z * z, k);
}

template <int kAct>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (kAct == TPK_ACT_SILU) return z * sigmoid_of(z);
  if constexpr (kAct == TPK_ACT_GELU) {
    float q, e;
    tail_of(z, q, e);
    const float h = q == 0.f ? 0.f : 0.5f * z * q;   // (an infinite z has no product with 0)
    return z > 0.f ? z - h : h;
  }
  if constexpr (kAct == TPK_ACT_GELU_TANH) return z * sigmoid_of(tanh_arg(z));
  return z;
}

// act(z), and its derivative in `slope`.
template <int kAct>
__device__ __forceinline__ float act_slope(float z, float& slope) {
  if constexpr (kAct == TPK_ACT_SILU) {
    const float s = sigmoid_of(z);
    slope = s * fmaf(z, 1.f - s, 1.f);
    return z * s;
  }
  if constexpr (kAct == TPK_ACT_GELU) {
    float q, e;
    tail_of(z, q, e);
    const float h = 0.5f * q, phi = z > 0.f ? 1.f - h : h;
    slope = fmaf(z * e, 0.39894228040143268f, phi);   // 1 / sqrt(2 pi)
    return z * phi;
  }
  if constexpr (kAct == TPK_ACT_GELU_TANH) {
    const float s = sigmoid_of(tanh_arg(z)), t = s * (1.f - s);
    constexpr float k = 1.5957691216057308f;
    slope = t == 0.f ? s : fmaf(z * t, fmaf(3.f * 0.044715f * k, z * z, k), s);   // far out z^2 has no value
    return z * s;
  }
  slope = 1.f;
  return z;
}

// body(integral_constant<act>): one copy of an epilogue's arithmetic per activation.
template <int kAct>
struct ActTag {
  static constexpr int value = kAct;
};
template <typename Body>
__device__ __forceinline__ void with_act(int act, Body body) {
  switch (act) {
    case TPK_ACT_SILU: body(ActTag<TPK_ACT_SILU>{}); break;
    case TPK_ACT_GELU: body(ActTag<TPK_ACT_GELU>{}); break;
    case TPK_ACT_GELU_TANH: body(ActTag<TPK_ACT_GELU_TANH>{}); break;
    default: body(ActTag<TPK_ACT_NONE>{}); break;
  }
}

}  // namespace tpk
