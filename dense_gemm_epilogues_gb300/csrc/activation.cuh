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
// exponential.  Two numbers at a time (paired FMAs): about 11 issue slots and two special
// functions each, where erfcf takes four times as many: the epilogue of a product of short
// depth would no longer hide behind its MMAs, nor the gradient's pass behind its loads.
// Exponentials and quotients are the hardware's (2 steps of fp32).  All keep NaN.
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

// Two fp32 numbers in one register pair, for the paired FMA.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t v;
  asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  return v;
}
__device__ __forceinline__ void split_pair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t both(float a) { return pair_of(a, a); }

// The normal distribution at x and y: p, q; e = exp(-x^2 / 2), exp(-y^2 / 2).
__device__ __forceinline__ void normal_pair(float x, float y, float& p, float& q, uint64_t& e) {
  const uint64_t k = pair_of(rcp_fast(fmaf(0.35f, fabsf(x), 1.0f)), rcp_fast(fmaf(0.35f, fabsf(y), 1.0f)));
  const uint64_t z = pair_of(x, y);
  float a, b;
  split_pair(mul_pair(mul_pair(both(-0.5f * LOG2_E), z), z), a, b);
  e = pair_of(exp2_fast(a), exp2_fast(b));
  uint64_t v = fma_pair(both(-0.0285310932f), k, both(0.1412722766f));
  v = fma_pair(v, k, both(-0.2507375181f));
  v = fma_pair(v, k, both(0.1541662067f));
  v = fma_pair(v, k, both(-0.0201176628f));
  v = fma_pair(v, k, both(0.1044274792f));
  v = fma_pair(v, k, both(0.1200617179f));
  v = fma_pair(v, k, both(0.1398360431f));
  v = fma_pair(v, k, both(0.1396225840f));
  split_pair(mul_pair(mul_pair(v, k), e), a, b);   // the distribution at -|x|, -|y|
  p = x < 0.0f ? a : 1.0f - a;
  q = y < 0.0f ? b : 1.0f - b;
}

constexpr float TANH_A = 1.5957691216057308f;   // 2 sqrt(2 / pi)

// Activations but GELU, which takes two numbers at a time.
template <int ACT>
__device__ __forceinline__ float activate_one(float x) {
  if constexpr (ACT == ACT_RELU) {
    float y;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(x));
    return y;
  } else if constexpr (ACT == ACT_GELU_TANH) {
    return x * sigmoid_fast(TANH_A * x * fmaf(0.044715f * x, x, 1.0f));
  } else if constexpr (ACT == ACT_SILU) {
    return x * sigmoid_fast(x);
  } else {
    return x;
  }
}

// x within +-16, beyond which the derivatives of both GELUs are 1 or 0 (and where x^2 would
// overflow far out); keeps NaN.
__device__ __forceinline__ float clamp16(float x) {
  float c;
  asm("max.NaN.f32 %0, %1, 0fC1800000;" : "=f"(c) : "f"(x));
  asm("min.NaN.f32 %0, %1, 0f41800000;" : "=f"(c) : "f"(c));
  return c;
}

// Their derivatives.
template <int ACT>
__device__ __forceinline__ float activate_grad_one(float x) {
  if constexpr (ACT == ACT_RELU) {
    return x > 0.0f ? 1.0f : x <= 0.0f ? 0.0f : x;
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float c = clamp16(x);
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

// x[i] = act(x[i]);  g[i] *= act'(z[i]).
template <int ACT, int N>
__device__ __forceinline__ void activate(float (&x)[N]) {
  static_assert(N % 2 == 0, "");
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (ACT == ACT_GELU) {
      float p, q;
      uint64_t e;
      normal_pair(x[i], x[i + 1], p, q, e);
      x[i] *= p;
      x[i + 1] *= q;
    } else {
      x[i] = activate_one<ACT>(x[i]);
      x[i + 1] = activate_one<ACT>(x[i + 1]);
    }
  }
}
template <int ACT, int N>
__device__ __forceinline__ void activate_grad(const float (&z)[N], float (&g)[N]) {
  static_assert(N % 2 == 0, "");
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    if constexpr (ACT == ACT_GELU) {
      float p, q;
      uint64_t e;
      const float a = clamp16(z[i]), b = clamp16(z[i + 1]);
      normal_pair(a, b, p, q, e);
      const uint64_t d = fma_pair(mul_pair(pair_of(a, b), both(0.3989422804f)), e, pair_of(p, q));
      split_pair(mul_pair(d, pair_of(g[i], g[i + 1])), g[i], g[i + 1]);
    } else {
      g[i] *= activate_grad_one<ACT>(z[i]);
      g[i + 1] *= activate_grad_one<ACT>(z[i + 1]);
    }
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
