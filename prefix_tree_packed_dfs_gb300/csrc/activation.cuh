// Activations of the projections and the feed-forward block, and their
// derivatives, in fp32 on packed pairs (include/tpk.h, TPK_ACT_*).
//   silu       z s,  s = 1 / (1 + e^-z)            s + z s (1 - s)
//   gelu       z Phi(z)                            Phi(z) + z phi(z)
//   gelu_tanh  z s(k (z + c z^3)), k = 2 sqrt(2 / pi), c = 0.044715
//              (0.5 (1 + tanh t) = s(2 t): no difference of close numbers)
// Phi through erfc(x) ~ (a1 t + .. + a5 t^5) e^{-x^2}, t = 1 / (1 + p x), for
// x >= 0 (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26), at a
// third of the instructions of the full-precision function, and the derivative
// shares the exponential.  Its error is absolute, 1.5e-7.  Below 0 Phi is half of
// that value itself, not 1 less the other half, so that gelu's tail keeps the fit's
// relative error: 5e-4 at z = -4, 1.6e-3 at -5 (a bf16 rounding is 2e-3 to 4e-3),
// 6.5e-3 at -7, where gelu is -9e-12.  (As 0.5 - w it was 4% off at -5.)
// An epilogue does 32,768 of these per tile and CTA while the tensor pipe needs
// 256 cycles per 64 elements of K, so instructions count: two values per
// instruction wherever there is a packed form.
#pragma once
#include "ptx.cuh"
#include "tpk.h"

namespace tpk {

constexpr float kActLog2e = 1.4426950408889634f;
constexpr float kTanhK = 1.5957691216057308f;   // 2 sqrt(2 / pi)

__device__ __forceinline__ uint64_t both(float v) { return ptx::f2(v, v); }
__device__ __forceinline__ uint64_t ex2_2(uint64_t v) {
  float a, b;
  ptx::unf2(v, a, b);
  return ptx::f2(ptx::ex2(a), ptx::ex2(b));
}
__device__ __forceinline__ uint64_t rcp_2(uint64_t v) {
  float a, b;
  ptx::unf2(v, a, b);
  return ptx::f2(ptx::rcp(a), ptx::rcp(b));
}
__device__ __forceinline__ uint64_t sigmoid_2(uint64_t z) {
  return rcp_2(ptx::add2(ex2_2(ptx::mul2(z, both(-kActLog2e))), both(1.f)));
}
// k (z + c z^3)
__device__ __forceinline__ uint64_t tanh_arg_2(uint64_t z, uint64_t zz) {
  return ptx::mul2(z, ptx::fma2(zz, both(0.044715f * kTanhK), both(kTanhK)));
}
// h below 0, 1 - h from there on.
__device__ __forceinline__ float side(float z, float h) {
  asm("{\n .reg .pred p;\n setp.ge.f32 p, %1, 0f00000000;\n @p sub.f32 %0, 0f3F800000, %0;\n}\n" : "+f"(h) : "f"(z));
  return h;
}
// Phi(z); e^{-z^2 / 2} in e
__device__ __forceinline__ uint64_t phi_2(uint64_t z, uint64_t& e) {
  constexpr uint64_t kSign = 0x8000000080000000ull;
  const uint64_t x = z & ~kSign;
  const uint64_t t = rcp_2(ptx::fma2(x, both(0.3275911f * 0.70710678118654752f), both(1.f)));
  e = ex2_2(ptx::mul2(ptx::mul2(z, z), both(-0.5f * kActLog2e)));
  uint64_t p = ptx::fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
  p = ptx::fma2(t, p, both(0.5f * 1.421413741f));
  p = ptx::fma2(t, p, both(0.5f * -0.284496736f));
  p = ptx::fma2(t, p, both(0.5f * 0.254829592f));
  float zl, zh, lo, hi;
  ptx::unf2(z, zl, zh);
  ptx::unf2(ptx::mul2(ptx::mul2(p, t), e), lo, hi);               // erfc(|z| / sqrt 2) / 2
  return ptx::f2(side(zl, lo), side(zh, hi));
}
// A square that a factor of zero may meet: finite.
__device__ __forceinline__ uint64_t square_2(uint64_t z) {
  float a, b;
  ptx::unf2(ptx::mul2(z, z), a, b);
  return ptx::f2(fminf(a, 1e36f), fminf(b, 1e36f));
}

template <int kAct>
__device__ __forceinline__ uint64_t act_2(uint64_t z) {
  if constexpr (kAct == TPK_ACT_SILU) return ptx::mul2(z, sigmoid_2(z));
  if constexpr (kAct == TPK_ACT_GELU) {
    uint64_t e;
    return ptx::mul2(z, phi_2(z, e));
  }
  if constexpr (kAct == TPK_ACT_GELU_TANH) return ptx::mul2(z, sigmoid_2(tanh_arg_2(z, ptx::mul2(z, z))));
  return z;
}

// act(z), and its derivative in `slope`.
template <int kAct>
__device__ __forceinline__ uint64_t act_slope_2(uint64_t z, uint64_t& slope) {
  const uint64_t one = both(1.f), minus = both(-1.f);
  if constexpr (kAct == TPK_ACT_SILU) {
    const uint64_t s = sigmoid_2(z), v = ptx::mul2(z, s);
    slope = ptx::fma2(v, ptx::fma2(s, minus, one), s);
    return v;
  }
  if constexpr (kAct == TPK_ACT_GELU) {
    uint64_t e;
    const uint64_t phi = phi_2(z, e);
    slope = ptx::fma2(ptx::mul2(z, e), both(0.39894228040143268f), phi);   // 1 / sqrt(2 pi)
    return ptx::mul2(z, phi);
  }
  if constexpr (kAct == TPK_ACT_GELU_TANH) {
    const uint64_t zz = square_2(z);
    const uint64_t s = sigmoid_2(tanh_arg_2(z, zz)), v = ptx::mul2(z, s);
    const uint64_t d = ptx::fma2(zz, both(3.f * 0.044715f * kTanhK), both(kTanhK));
    slope = ptx::fma2(ptx::mul2(v, ptx::fma2(s, minus, one)), d, s);
    return v;
  }
  slope = one;
  return z;
}

// body(tag of the activation): one copy of an epilogue's arithmetic per activation.
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
