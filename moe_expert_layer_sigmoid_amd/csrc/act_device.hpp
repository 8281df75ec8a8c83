// Activations and their derivatives in f32, shared by the quantiser behind
// SwiGLU, the products' epilogues and the gradient through them.
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

#include "gelu_tail.hpp"

namespace moe {

// e^-g from the hardware's exp2 (1 ulp), its argument carried in two parts:
// one f32 product -g log2(e) would lose log2|g| bits of the result.
__device__ __forceinline__ float exp_neg(float g) {
  const float hi = g * -1.44269504f;
  const float lo = fmaf(g, -1.44269504f, -hi) + g * -1.92596299e-8f;  // log2(e) = 1.44269504 + 1.92596299e-8
  return __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.69314718f, 1.0f);
}

// silu(g) u for g >= kFarGate: the hardware's reciprocal (1 ulp) in place of a
// division keeps the kernel on the memory's side of its balance (in all within
// 9 x 2^-24 of the value, far below the codes' 2^-4).  Above 88 the sigmoid
// rounds to 1, and e^-inf by the two parts above would be NaN.
constexpr float kFarGate = -80.0f;
__device__ __forceinline__ float silu_mul(float g, float u) {
  const float e = exp_neg(g);
  const float r = g > 88.0f ? 1.0f : __builtin_amdgcn_rcpf(1.0f + e);
  return g * r * u;
}

// silu(g) u for g < kFarGate, where 1 + e^-g rounds to e^-g: g e^g u.  Below
// -87 neither e^g nor its reciprocal is a normal f32, while the product may be
// one (silu(-88) = -5e-37, times u): t = e^(g/4) is normal down to -349, where
// no u brings the product back into range, and every partial product is
// normal wherever the result is (four errors of t and five roundings: 21 x
// 2^-24).  g = -inf: NaN, as in the formula.
__device__ __forceinline__ float silu_mul_far(float g, float u) {
  const float t = exp_neg(-0.25f * g);
  return (g * t) * (u * t) * t * t;
}

// moe_act_t of include/moe.h
enum { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4, kActs = 5 };

constexpr float kGeluC = 0.797884561f;  // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

// Phi(-a) e^(a^2 / 2) for a >= 0 (gelu_tail.hpp).  One exponential then gives Phi and phi
// both, and the negative tail keeps its relative error.  (erfcf bound the gradient by its
// arithmetic: 29343 rows x 672, 46 us for 31.)
__device__ __forceinline__ float scaled_tail(float a) {
  const float t = __builtin_amdgcn_rcpf(fmaf(kTailArg, a, 1.0f));
  float q = kTail[kTailDegree];
#pragma unroll
  for (int i = kTailDegree - 1; i >= 0; --i) q = fmaf(q, t, kTail[i]);
  return t * q;
}
// e^(-z^2 / 2) for z >= -13 and beyond any normal value above
__device__ __forceinline__ float gauss(float z) {
  const float h = 0.5f * z * z;
  return exp_neg(h > 100.0f ? 100.0f : h);
}
constexpr float kFarGelu = -13.0f;
constexpr float kPhi0 = 0.398942280f;  // 1 / sqrt(2 pi)
// e^(-x^2 / 8) for z < kFarGelu, x = z no lower than -27, where its fourth power is zero
__device__ __forceinline__ float gauss_root(float& x) {
  x = x < -27.0f ? -27.0f : x;
  return exp_neg(0.125f * x * x);
}

// Where the exponentials of act or act' leave f32's normal range while a product with
// them may not: the far forms below, e^t in four factors.
template <int ACT>
constexpr float far_below() {
  return ACT == kActSilu ? kFarGate : ACT == kActGelu ? kFarGelu : ACT == kActGeluTanh ? -9.0f : -__builtin_inff();
}

// act(g) u.  gelu: z Phi(z); gelu_tanh: 0.5 z (1 + tanh w) = z sigmoid(2 w) with
// w = sqrt(2 / pi) (z + 0.044715 z^3).  The exponent's own rounding grows with it:
// relative errors of up to (8 + z^2) 2^-23 (gelu) and (8 + |2 w|) 2^-22 (gelu_tanh).
template <int ACT>
__device__ __forceinline__ float act_near(float g, float u) {  // g >= far_below<ACT>(), or NaN
  if constexpr (ACT == kActRelu) return (g < 0.0f ? 0.0f : g) * u;
  else if constexpr (ACT == kActSilu) return silu_mul(g, u);
  else if constexpr (ACT == kActGelu) {
    const float s = scaled_tail(fabsf(g)) * gauss(g);
    return g * (g < 0.0f ? s : 1.0f - s) * u;
  }
  else if constexpr (ACT == kActGeluTanh) {
    const float t = 2.0f * kGeluC * g * fmaf(kGeluA * g, g, 1.0f);
    return g * (t > 88.0f ? 1.0f : __builtin_amdgcn_rcpf(1.0f + exp_neg(t))) * u;
  }
  else return g * u;
}
template <int ACT>
__device__ __forceinline__ float act_far(float g, float u) {  // g < far_below<ACT>()
  if constexpr (ACT == kActSilu) return silu_mul_far(g, u);
  else if constexpr (ACT == kActGelu) {
    float x = g;
    const float t = gauss_root(x);
    return (g * scaled_tail(-x) * t) * (u * t) * t * t;
  }
  else {  // gelu_tanh: e^(2 w); below -400 every factor is zero
    const float t = 2.0f * kGeluC * g * fmaf(kGeluA * g, g, 1.0f), s = exp_neg(t < -400.0f ? 100.0f : -0.25f * t);
    return (g * s) * (u * s) * s * s;
  }
}
// v = act(g) u of V values, with one branch for all that are far: no trained model's
// get there, and a branch a value would run their exponentials one after the other
// (gelu, 1295 x 3840, K 104, with bias, residual and z, bf16: 18.3 us for 20.2).
template <int ACT, int V>
__device__ __forceinline__ void act_row(const float (&g)[V], const float (&u)[V], float (&v)[V]) {
  bool far = false;
#pragma unroll
  for (int e = 0; e < V; ++e) {
    v[e] = act_near<ACT>(g[e], u[e]);
    far |= g[e] < far_below<ACT>();
  }
  if constexpr (ACT == kActSilu || ACT == kActGelu || ACT == kActGeluTanh) {
    if (far) {
#pragma unroll
      for (int e = 0; e < V; ++e)
        if (g[e] < far_below<ACT>()) v[e] = act_far<ACT>(g[e], u[e]);
    }
  }
}
// ... of V gates and values, or (G = 1) of V values alone
template <int ACT, int G, int V>
__device__ __forceinline__ void act_gated(const float (&z)[G][V], float (&v)[V]) {
  float u[V];
#pragma unroll
  for (int e = 0; e < V; ++e) u[e] = G == 2 ? z[G - 1][e] : 1.0f;
  act_row<ACT>(z[0], u, v);
}

// act(z) and act'(z) together, from one exponential:
//  silu:      s = sigmoid(z): z s and s (1 + z (1 - s)), 1 - s = e s
//  gelu:      z Phi(z) and Phi(z) + z phi(z)
//  gelu_tanh: s = sigmoid(t), t = 2 w: z s and s + z s (1 - s) t'(z); beyond 16 the
//             slope is 1 or 0 in f32, and t' would overflow
// An infinite z gives NaN where the formula has 0 times infinity (z phi(z), z (1 - s)).
// For z >= far_below<ACT>(); below: grad_far.
template <int ACT>
__device__ __forceinline__ void act_slope(float z, float& f, float& d) {
  if constexpr (ACT == kActRelu) {
    f = z < 0.0f ? 0.0f : z;
    d = z <= 0.0f ? 0.0f : 1.0f;
  } else if constexpr (ACT == kActSilu) {
    const float e = z > 88.0f ? 0.0f : exp_neg(z), s = __builtin_amdgcn_rcpf(1.0f + e);
    f = z * s;
    d = s * fmaf(z, e * s, 1.0f);
  } else if constexpr (ACT == kActGelu) {
    const float w = gauss(z), s = scaled_tail(fabsf(z)) * w, c = z < 0.0f ? s : 1.0f - s;
    f = z * c;
    d = fmaf(z, kPhi0 * w, c);
  } else if constexpr (ACT == kActGeluTanh) {
    const float x = z > 16.0f ? 16.0f : z < -16.0f ? -16.0f : z;
    const float x2 = x * x, t = 2.0f * kGeluC * x * fmaf(kGeluA, x2, 1.0f);
    const float e = t > 88.0f ? 0.0f : exp_neg(t < -80.0f ? -80.0f : t), s = __builtin_amdgcn_rcpf(1.0f + e);
    f = z * s;
    d = s * fmaf(z * (e * s), 2.0f * kGeluC * fmaf(3.0f * kGeluA, x2, 1.0f), 1.0f);
  } else {
    f = z;
    d = 1.0f;
  }
}
// dz and df for z < far_below<ACT>(): v act'(z) and w act(z), e^t in four factors
// (silu: act' = e^z (1 + z); gelu: e^(-z^2 / 2) (scaled tail + z / sqrt(2 pi));
// gelu_tanh: e^t (1 + z t'(z)); 1 - s is 1 there).  z - z: both are NaN for z = -inf,
// which the bounds on x hide (silu's t is 0 there, and 0 times z is NaN already).
template <int ACT>
__device__ __forceinline__ void grad_far(float z, float v, float w, float& dz, float& df) {
  if constexpr (ACT == kActSilu) {
    const float t = exp_neg(z < -400.0f ? 100.0f : -0.25f * z);
    dz = ((1.0f + z) * t) * (v * t) * t * t;
    df = (z * t) * (w * t) * t * t;
  } else if constexpr (ACT == kActGelu) {
    float x = z;
    const float t = gauss_root(x), c = scaled_tail(-x);
    dz = (fmaf(x, kPhi0, c) * t) * (v * t) * t * t + (z - z);
    df = (x * c * t) * (w * t) * t * t + (z - z);
  } else if constexpr (ACT == kActGeluTanh) {
    const float x = z < -20.0f ? -20.0f : z, x2 = x * x;  // t(-20) = -603: zero
    const float t = exp_neg(-0.5f * kGeluC * x * fmaf(kGeluA, x2, 1.0f));
    dz = (fmaf(x * 2.0f * kGeluC, fmaf(3.0f * kGeluA, x2, 1.0f), 1.0f) * t) * (v * t) * t * t + (z - z);
    df = (x * t) * (w * t) * t * t + (z - z);
  }
}

// f(std::integral_constant<int, act>) for a runtime act.
template <class F>
__host__ __device__ __forceinline__ void with_act(int act, F f) {
  if (act == kActSilu) f(std::integral_constant<int, kActSilu>{});
  else if (act == kActRelu) f(std::integral_constant<int, kActRelu>{});
  else if (act == kActGelu) f(std::integral_constant<int, kActGelu>{});
  else if (act == kActGeluTanh) f(std::integral_constant<int, kActGeluTanh>{});
  else f(std::integral_constant<int, kActNone>{});
}

}  // namespace moe
