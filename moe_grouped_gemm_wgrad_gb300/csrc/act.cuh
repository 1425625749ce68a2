// Activations of the expert products and their slopes, in fp32.
//   relu(x) = max(x, 0), slope 0 at 0
//   gelu(x) = x Phi(x), Phi the normal distribution function; slope Phi(x) + x phi(x)
//   silu(x) = x s(x), s the logistic function; slope s(x) (1 + x (1 - s(x)))
//   swiglu, geglu: silu or gelu of the gate times the up value (two halves of the product's
//   columns: gate first)
#pragma once
#include <cuda_runtime.h>

namespace mgw {

constexpr int kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4, kActGeglu = 5;

__host__ __device__ constexpr bool act_gated(int act) { return act == kActSwiglu || act == kActGeglu; }
// The activation applied to the gate (or to the only value).
__host__ __device__ constexpr int act_inner(int act) {
  return act == kActSwiglu ? kActSilu : act == kActGeglu ? kActGelu : act;
}

__device__ __forceinline__ float ex2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The lower tail h = Phi(-|x|) of the normal distribution and e = exp(-x^2 / 2), by formula
// 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions: erfc(u) =
// (a1 t + .. + a5 t^5) exp(-u^2), t = 1 / (1 + 0.3275911 u), with |error| <= 1.5e-7 in erf.
// Every caller rounds to bf16 (half an ulp is 2e-3 of the value), or sums such values; x Phi(x)
// is off by at most 1e-7 max(|x|, 1), as it would be through 0.5 + 0.5 erf.
__device__ __forceinline__ float normal_tail(float x, float& e) {
  const float t = rcp_approx(fmaf(0.3275911f * 0.70710678f, fabsf(x), 1.0f));
  const float y = 0.84932180028801907f * x;  // sqrt(log2(e) / 2)
  e = ex2_approx(-y * y);
  float p = fmaf(0.5f * 1.061405429f, t, 0.5f * -1.453152027f);
  p = fmaf(p, t, 0.5f * 1.421413741f);
  p = fmaf(p, t, 0.5f * -0.284496736f);
  p = fmaf(p, t, 0.5f * 0.254829592f);
  return p * t * e;
}

// 1 / (1 + e^-x); e^-x may overflow to infinity, whose reciprocal is 0.
__device__ __forceinline__ float logistic_fast(float x) {
  return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
}

// x Phi(x) = max(x, 0) - |x| h, with |x| bounded so that an infinite x meets h = 0 as a number.
__device__ __forceinline__ float gelu_from_tail(float x, float h) {
  return fmaf(-fminf(fabsf(x), 1e30f), h, fmaxf(x, 0.0f));
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActRelu) return x <= 0.0f ? 0.0f : x;  // NaN stays NaN
  if constexpr (ACT == kActGelu) {
    float e;
    return gelu_from_tail(x, normal_tail(x, e));
  }
  if constexpr (ACT == kActSilu) return x * logistic_fast(x);
  return x;
}

// Value and slope together (the backward pass of a gated activation needs both).
template <int ACT>
__device__ __forceinline__ void act_value_slope(float x, float& value, float& slope) {
  if constexpr (ACT == kActRelu) {
    value = x <= 0.0f ? 0.0f : x;
    slope = x > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActGelu) {
    float e;
    const float h = normal_tail(x, e);
    value = gelu_from_tail(x, h);
    slope = fmaf(0.3989422804014327f * x, e, x >= 0.0f ? 1.0f - h : h);  // Phi(x) + x phi(x)
  } else if constexpr (ACT == kActSilu) {
    const float s = logistic_fast(x);
    value = x * s;
    slope = fmaf(value, 1.0f - s, s);
  } else {
    value = x;
    slope = 1.0f;
  }
}

}  // namespace mgw
