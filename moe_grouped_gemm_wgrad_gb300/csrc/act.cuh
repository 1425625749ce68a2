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

__device__ __forceinline__ float normal_cdf(float x) {
  return 0.5f + 0.5f * erff(x * 0.70710678118654752f);
}

// 1 / (1 + e^-x) from e^-|x|, which cannot overflow.  The results are rounded to bf16 by
// every caller in the GEMM path, so the fast exponential and division (a few fp32 ulp) do.
__device__ __forceinline__ float logistic_fast(float x) {
  const float q = __expf(-fabsf(x));
  const float r = __fdividef(1.0f, 1.0f + q);
  return x >= 0.0f ? r : q * r;
}

template <int ACT>
__device__ __forceinline__ float act_value(float x) {
  if constexpr (ACT == kActRelu) return fmaxf(x, 0.0f);
  if constexpr (ACT == kActGelu) return x * normal_cdf(x);
  if constexpr (ACT == kActSilu) return x * logistic_fast(x);
  return x;
}

// Value and slope together (the backward pass of a gated activation needs both).
template <int ACT>
__device__ __forceinline__ void act_value_slope(float x, float& value, float& slope) {
  if constexpr (ACT == kActRelu) {
    value = fmaxf(x, 0.0f);
    slope = x > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (ACT == kActGelu) {
    const float cdf = normal_cdf(x);
    value = x * cdf;
    slope = cdf + x * (0.3989422804014327f * __expf(-0.5f * x * x));
  } else if constexpr (ACT == kActSilu) {
    const float s = logistic_fast(x);
    value = x * s;
    slope = s + value * (1.0f - s);
  } else {
    value = x;
    slope = 1.0f;
  }
}

}  // namespace mgw
