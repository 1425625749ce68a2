// Activations of the expert products and their slopes, in fp32.
//   relu(x) = max(x, 0), slope 0 at 0; NaN has neither a value nor a slope
//   gelu(x) = x Phi(x), Phi the normal distribution function; slope Phi(x) + x phi(x)
//   silu(x) = x s(x), s the logistic function; slope s(x) (1 + x (1 - s(x)))
//   swiglu, geglu: silu or gelu of the gate times the up value (two halves of the product's
//   columns: gate first)
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

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

// 1 / (1 + e^-x); e^-x may overflow to infinity, whose reciprocal is 0.
__device__ __forceinline__ float logistic_fast(float x) {
  return rcp_approx(1.0f + ex2_approx(-1.4426950408889634f * x));
}

// Activations other than the GELU, which comes in pairs only (act_value2).
template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  static_assert(ACT != kActGelu, "act_value2");
  if constexpr (ACT == kActRelu) return x <= 0.0f ? 0.0f : x;  // NaN stays NaN
  if constexpr (ACT == kActSilu) return x * logistic_fast(x);
  return x;
}

// Two packed fp32 values per instruction (the FMA pipe's packed form).
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(F2 a, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a.v));
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// Of two values: minus the lower tail h = Phi(-|x|) of the normal distribution, and e = exp(-x^2 / 2),
// by formula 7.1.26 of Abramowitz and Stegun, Handbook of Mathematical Functions: erfc(u) =
// (a1 t + .. + a5 t^5) exp(-u^2), t = 1 / (1 + 0.3275911 u), with |error| <= 1.5e-7 in erf (the
// polynomial has its signs turned).  In fp32 x Phi(x) is off by up to 1.6e-7 max(|x|, 1), where
// x (0.5 + 0.5 erf) is by 1.1e-7, and the slope by 6.6e-8 rms over normal x, where that is by 2.7e-8.
// Next to bf16 (half an ulp is up to 2^-8 of a value) that is nothing, and far below x = 0 the tail
// is the better of the two; the one fp32 output that has it in is the bias gradient, a sum of slopes.
__device__ __forceinline__ F2 minus_tail2(float x0, float x1, F2& e) {
  const float t0 = rcp_approx(fmaf(0.3275911f * 0.70710678f, fabsf(x0), 1.0f));
  const float t1 = rcp_approx(fmaf(0.3275911f * 0.70710678f, fabsf(x1), 1.0f));
  const F2 x = f2(x0, x1), t = f2(t0, t1);
  float e0, e1;
  split(mul2(mul2(x, x), f2(-0.72134752044448170f, -0.72134752044448170f)), e0, e1);  // -log2(e) / 2
  e = f2(ex2_approx(e0), ex2_approx(e1));
  F2 p = fma2(f2(-0.5f * 1.061405429f, -0.5f * 1.061405429f), t, f2(0.5f * 1.453152027f, 0.5f * 1.453152027f));
  p = fma2(p, t, f2(-0.5f * 1.421413741f, -0.5f * 1.421413741f));
  p = fma2(p, t, f2(0.5f * 0.284496736f, 0.5f * 0.284496736f));
  p = fma2(p, t, f2(-0.5f * 0.254829592f, -0.5f * 0.254829592f));
  return mul2(mul2(p, t), e);
}
// x Phi(x) = max(x, 0) - |x| h, with |x| bounded so that an infinite x meets h = 0 as a number.
__device__ __forceinline__ F2 gelu2_from_tail(float x0, float x1, F2 minus_h) {
  return fma2(f2(fminf(fabsf(x0), 1e30f), fminf(fabsf(x1), 1e30f)), minus_h,
              f2(fmaxf(x0, 0.0f), fmaxf(x1, 0.0f)));
}

// act_value of two values in place.  The GELU's polynomial and products run packed: of some 28
// instructions a pair about 20 are left.
template <int ACT>
__device__ __forceinline__ void act_value2(float& x0, float& x1) {
  if constexpr (ACT == kActGelu) {
    F2 e;
    const F2 p = minus_tail2(x0, x1, e);
    split(gelu2_from_tail(x0, x1, p), x0, x1);
  } else {
    x0 = act_value<ACT>(x0);
    x1 = act_value<ACT>(x1);
  }
}

// Value and slope together (the backward pass of a gated activation needs both).
template <int ACT>
__device__ __forceinline__ void act_value_slope(float x, float& value, float& slope) {
  static_assert(ACT != kActGelu, "act_value_slope2");
  if constexpr (ACT == kActRelu) {
    value = x <= 0.0f ? 0.0f : x;
    slope = x > 0.0f ? 1.0f : x <= 0.0f ? 0.0f : x;  // NaN stays NaN
  } else if constexpr (ACT == kActSilu) {
    const float s = logistic_fast(x);
    value = x * s;
    slope = fmaf(value, 1.0f - s, s);
  } else {
    value = x;
    slope = 1.0f;
  }
}

// act_value_slope of two values.
template <int ACT>
__device__ __forceinline__ void act_value_slope2(float x0, float x1, float (&value)[2], float (&slope)[2]) {
  if constexpr (ACT == kActGelu) {
    F2 e;
    const F2 p = minus_tail2(x0, x1, e);
    split(gelu2_from_tail(x0, x1, p), value[0], value[1]);
    float p0, p1;
    split(p, p0, p1);
    const F2 cdf = f2(x0 >= 0.0f ? 1.0f + p0 : -p0, x1 >= 0.0f ? 1.0f + p1 : -p1);
    const F2 phi = mul2(f2(x0, x1), f2(0.3989422804014327f, 0.3989422804014327f));
    split(fma2(phi, e, cdf), slope[0], slope[1]);  // Phi(x) + x phi(x)
  } else {
    act_value_slope<ACT>(x0, value[0], slope[0]);
    act_value_slope<ACT>(x1, value[1], slope[1]);
  }
}

}  // namespace mgw
