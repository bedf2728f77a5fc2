// activation.cuh -- activations of fully connected layers and their derivatives (internal).
//
//   gelu       x P(x),  P the normal distribution;   its derivative P(x) + x p(x)
//   gelu_tanh  x s(2 u),  u = sqrt(2 / pi) (x + 0.044715 x^3),  s(v) = 1 / (1 + exp(-v)):
//              the same as 0.5 x (1 + tanh u), without its cancellation for negative x
//   silu       x s(x)
//
// P(-t) = exp(-t^2 / 2) R(t) for t >= 0, and R(t) = k Q(k) with k = 1 / (1 + 0.35 t): the
// substitution makes R, which falls from 1/2 like 1 / t, smooth up to k = 0.  Q of degree 8
// was fitted here to erfcx by weighted least squares; in fp32 P is off by at most 2.3e-7, and
// by 9e-7 of its value down to x = -4 (3.4e-6 at -9).  The derivative needs the same
// exponential.  About 18 instructions, of which two on the special function unit, where
// erfcf takes twice as many: the epilogue of a product of short depth would no longer hide
// behind its MMAs.  Exponentials and quotients are the hardware's (2 steps of fp32).  All
// keep NaN.
#pragma once

#include "common.cuh"

namespace gemmlib {

enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };   // gemm_linear_act_t

#if defined(__CUDACC__)

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
constexpr float LOG2_E = 1.4426950408889634f;

// 1 / (1 + exp(-v))
__device__ __forceinline__ float sigmoid_fast(float v) { return rcp_fast(1.0f + exp2_fast(-LOG2_E * v)); }

// The normal distribution at x; e = exp(-x^2 / 2).
__device__ __forceinline__ float normal_fast(float x, float& e) {
  const float k = rcp_fast(fmaf(0.35f, fabsf(x), 1.0f));
  e = exp2_fast(-0.5f * LOG2_E * x * x);
  float q = fmaf(-0.0285310932f, k, 0.1412722766f);
  q = fmaf(q, k, -0.2507375181f);
  q = fmaf(q, k, 0.1541662067f);
  q = fmaf(q, k, -0.0201176628f);
  q = fmaf(q, k, 0.1044274792f);
  q = fmaf(q, k, 0.1200617179f);
  q = fmaf(q, k, 0.1398360431f);
  q = fmaf(q, k, 0.1396225840f);
  const float half = q * k * e;   // the distribution at -|x|
  return x < 0.0f ? half : 1.0f - half;
}

constexpr float TANH_A = 1.5957691216057308f;   // 2 sqrt(2 / pi)

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == ACT_RELU) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    return x * normal_fast(x, e);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    return x * sigmoid_fast(TANH_A * x * fmaf(0.044715f * x, x, 1.0f));
  } else if constexpr (ACT == ACT_SILU) {
    return x * sigmoid_fast(x);
  } else {
    return x;
  }
}

// The derivative at x.
template <int ACT>
__device__ __forceinline__ float activate_grad(float x) {
  if constexpr (ACT == ACT_RELU) {
    return x > 0.0f ? 1.0f : x <= 0.0f ? 0.0f : x;
  } else if constexpr (ACT == ACT_GELU) {
    float e;
    const float p = normal_fast(x, e);
    return fmaf(x * 0.3989422804f, e, p);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    // Beyond +-16 it is 1 or 0; x^2 would overflow far out.
    float c;
    asm("max.NaN.f32 %0, %1, 0fC1800000;" : "=f"(c) : "f"(x));
    asm("min.NaN.f32 %0, %1, 0f41800000;" : "=f"(c) : "f"(c));
    const float s = sigmoid_fast(TANH_A * c * fmaf(0.044715f * c, c, 1.0f));
    const float n = sigmoid_fast(-TANH_A * c * fmaf(0.044715f * c, c, 1.0f));   // 1 - s, without cancellation
    return fmaf(c * s * n, TANH_A * fmaf(0.134145f * c, c, 1.0f), s);
  } else if constexpr (ACT == ACT_SILU) {
    float c;
    asm("max.NaN.f32 %0, %1, 0fC2B00000;" : "=f"(c) : "f"(x));   // beyond +-88 it is 1 or 0
    asm("min.NaN.f32 %0, %1, 0f42B00000;" : "=f"(c) : "f"(c));
    const float s = sigmoid_fast(c);
    return s * fmaf(c, sigmoid_fast(-c), 1.0f);
  } else {
    return 1.0f;
  }
}

// f(tag) for an activation: f's argument has it as a constant `value`.
template <int V>
struct ActTag {
  static constexpr int value = V;
};
template <typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == ACT_NONE) f(ActTag<ACT_NONE>{});
  else if (act == ACT_RELU) f(ActTag<ACT_RELU>{});
  else if (act == ACT_GELU) f(ActTag<ACT_GELU>{});
  else if (act == ACT_GELU_TANH) f(ActTag<ACT_GELU_TANH>{});
  else f(ActTag<ACT_SILU>{});
}

#endif

}  // namespace gemmlib
