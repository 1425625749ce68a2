// Router: the top_k experts of every token and their weights, and the backward pass.
//
//   s = softmax(x) or logistic(x), 0 where x is -inf (an expert the token may not use)
//   v = x without a balance bias (both scores grow with x, so the order is that of the logits
//       and no rounding of the score can reorder or tie two experts), else s + bias
//   with groups: a group's value is its best v, or the sum of its best two (of s + bias, or
//       of s without a bias); the top_groups best groups stay
//   expert_idx = the top_k largest v, ties to the lower index; -1 when fewer are left
//   w_k = scale * s_k, renormalised: scale * s_k / sum_j s_j over the chosen
//
// One warp per token: lane l holds the V experts l V .. l V + V - 1 (E <= 32 V), so of equal
// values the lowest lane's is the lowest index.  Each of the top_k rounds is one warp-wide
// integer maximum (redux) over order-preserving keys, one ballot, and an update of the winning
// lane's V keys.  The renormalised softmax needs the chosen logits only; sums are fp32.
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;  // tokens per CTA

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Order-preserving map of a float (not NaN) to an unsigned integer; both zeros map alike.
// 0 is below every float's key and stands for "not available".
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}

// e^(x - m), exactly 1 at x == m (also when both are infinite)
__device__ __forceinline__ float exp_from(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// The logistic function and its complement from e^-|x|, which cannot overflow.
__device__ __forceinline__ void logistic(float x, float& s, float& c) {
  const float q = expf(-fabsf(x));
  const float r = 1.0f / (1.0f + q);
  s = x >= 0.0f ? r : q * r;
  c = x >= 0.0f ? q * r : r;
}

constexpr float kNegInf = -__builtin_huge_valf();

// Lane `lane`'s V logits, -inf past E; a NaN is reported and counts as -inf.
template <typename T, int V>
__device__ __forceinline__ void load_row(const T* row, int E, int lane, float (&x)[V], int* status) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    float v = e < E ? load_logit(row + e) : kNegInf;
    if (v != v) {
      nan = true;
      v = kNegInf;
    }
    x[j] = v;
  }
  if (nan && status != nullptr) atomicOr(status, kDevBadLogit);
}

// Scores of the row: softmax over the warp's logits, or the logistic function of each.
template <int V, bool SIGMOID>
__device__ __forceinline__ void row_scores(const float (&x)[V], float (&s)[V]) {
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float c;
      logistic(x[j], s[j], c);
    }
  } else {
    float m = kNegInf;
#pragma unroll
    for (int j = 0; j < V; ++j) m = fmaxf(m, x[j]);
    m = warp_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = x[j] == kNegInf ? 0.0f : exp_from(x[j], m);
      sum += s[j];
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] *= inv;
  }
}

template <typename T, int V, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
  extern __shared__ float s_vals[];  // with groups: kWarps rows of E values
  const int lane = static_cast<int>(lane_id());
  const int warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= a.T) return;
  const int E = a.E;
  float x[V], s[V];
  load_row<T, V>(static_cast<const T*>(a.logits) + t * E, E, lane, x, a.status);
  const bool need_scores = SIGMOID || !RENORM || a.scores != nullptr || a.bias != nullptr ||
                           (a.groups > 1 && a.group_best == 2);
  if (need_scores) row_scores<V, SIGMOID>(x, s);
  if (a.scores != nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane * V + j;
      if (e < E) a.scores[t * E + e] = s[j];
    }
  }
  uint32_t key[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    const float v = a.bias != nullptr && e < E ? s[j] + a.bias[e] : x[j];
    key[j] = x[j] == kNegInf ? 0u : key_of(v);
  }
  if (a.groups > 1) {
    // Group values through shared memory: lane g takes group g.
    const int per = E / a.groups;
    float* row = s_vals + warp * E;
    const bool sum2 = a.group_best == 2;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane * V + j;
      if (e < E) row[e] = key[j] == 0u ? kNegInf : (sum2 && a.bias == nullptr ? s[j] : value_of(key[j]));
    }
    __syncwarp();
    uint32_t gkey = 0;
    if (lane < a.groups) {
      float b1 = kNegInf, b2 = kNegInf;
      for (int i = 0; i < per; ++i) {
        const float v = row[lane * per + i];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      if (b1 != kNegInf) gkey = key_of(sum2 && b2 != kNegInf ? b1 + b2 : b1);
    }
    unsigned kept = 0;
    for (int i = 0; i < a.top_groups; ++i) {
      const uint32_t m = __reduce_max_sync(kAll, gkey);
      if (m == 0u) break;
      const int g = __ffs(__ballot_sync(kAll, gkey == m)) - 1;
      kept |= 1u << g;
      if (lane == g) gkey = 0u;
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int e = lane * V + j;
      if (e < E && !((kept >> (e / per)) & 1u)) key[j] = 0u;
    }
  }
  // lane k keeps the k-th choice
  int my_e = -1;
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) best = max(best, key[j]);
  for (int k = 0; k < a.top_k; ++k) {
    const uint32_t m = __reduce_max_sync(kAll, best);
    if (m == 0u) break;
    const int src = __ffs(__ballot_sync(kAll, best == m)) - 1;
    int pick = 0;
    if (lane == src) {
      bool found = false;
      best = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (!found && key[j] == m) {
          found = true;
          pick = j;
          key[j] = 0u;
        }
        best = max(best, key[j]);
      }
    }
    pick = __shfl_sync(kAll, pick, src) + src * V;
    if (lane == k) my_e = pick;
  }
  // weights of the chosen, from their logits or their scores
  float w = 0.0f, xk = kNegInf;
  if (my_e >= 0) xk = load_logit(static_cast<const T*>(a.logits) + t * E + my_e);
  if constexpr (SIGMOID) {
    float c;
    if (my_e >= 0) logistic(xk, w, c);
    if constexpr (RENORM) {
      const float sum = warp_sum(w);
      w = sum > 0.0f ? w / sum : 0.0f;
    }
  } else if constexpr (RENORM) {
    const float m = warp_max(xk);
    if (my_e >= 0) w = exp_from(xk, m);
    const float sum = warp_sum(w);
    w = sum > 0.0f ? w / sum : 0.0f;
  } else {
    // the score of expert my_e lives in lane my_e / V
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float v = __shfl_sync(kAll, s[j], my_e >= 0 ? my_e / V : 0);
      if (my_e >= 0 && my_e % V == j) w = v;
    }
  }
  if (lane < a.top_k) {
    a.expert_idx[t * a.top_k + lane] = my_e;
    a.weights[t * a.top_k + lane] = w * a.scale;
  }
}

// dlogits of one token per warp.  With G = dL/ds (the scores' own gradient plus the weights'):
// softmax dx = s (G - sum s G), logistic dx = G s (1 - s).  Renormalised weights w = scale * p
// depend on the chosen only: their part is p_k (g_k - sum_j p_j g_j), g = scale * dw, times
// (1 - s_k) for the logistic function.
template <typename T, int V, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteBwdArgs a) {
  extern __shared__ float s_add[];  // kWarps rows of E: the chosen experts' own terms
  const int lane = static_cast<int>(lane_id());
  const int warp = threadIdx.x >> 5;
  const long long t = static_cast<long long>(blockIdx.x) * kWarps + warp;
  if (t >= a.T) return;
  const int E = a.E;
  float* add = s_add + static_cast<size_t>(warp) * E;
  for (int e = lane; e < E; e += 32) add[e] = 0.0f;
  __syncwarp();
  const T* row = static_cast<const T*>(a.logits) + t * E;
  float x[V], s[V];
  load_row<T, V>(row, E, lane, x, a.status);
  const bool dense = !SIGMOID && (!RENORM || a.dscores != nullptr);
  if (dense || a.dscores != nullptr) row_scores<V, SIGMOID>(x, s);
  // the chosen experts' terms: added to G (plain softmax) or straight to dx (the others)
  if (a.dweights != nullptr) {
    int e = -1;
    float g = 0.0f;
    if (lane < a.top_k) {
      e = a.expert_idx[t * a.top_k + lane];
      if (e < -1 || e >= E) {
        if (a.status != nullptr) atomicOr(a.status, kDevBadIndex);
        e = -1;
      }
      if (e >= 0) g = a.dweights[t * a.top_k + lane] * a.scale;
    }
    float xk = e >= 0 ? load_logit(row + e) : kNegInf;
    if (xk != xk) xk = kNegInf;
    if (xk == kNegInf) e = -1, g = 0.0f;
    float term = g;
    if constexpr (RENORM) {
      float p = 0.0f, c = 1.0f;
      if constexpr (SIGMOID) {
        if (e >= 0) logistic(xk, p, c);
      } else {
        const float m = warp_max(xk);
        if (e >= 0) p = exp_from(xk, m);
      }
      const float sum = warp_sum(p);
      p = sum > 0.0f ? p / sum : 0.0f;
      term = p * (g - warp_sum(p * g));
      if constexpr (SIGMOID) term *= c;
    } else if constexpr (SIGMOID) {
      float p, c;
      logistic(xk, p, c);
      term = g * p * c;
    }
    if (e >= 0) atomicAdd(&add[e], term);  // experts of a token differ: one term each
    __syncwarp();
  }
  float G[V];
  float dot = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    float d = 0.0f;
    if (e < E && x[j] != kNegInf) {
      if (a.dscores != nullptr) d = a.dscores[t * E + e];
      if (!SIGMOID && !RENORM) d += add[e];
    }
    G[j] = d;
    if (dense) dot += s[j] * d;
  }
  if (dense) dot = warp_sum(dot);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = lane * V + j;
    if (e >= E) continue;
    float dx = 0.0f;
    if constexpr (SIGMOID) {
      if (a.dscores != nullptr) {
        float p, c;
        logistic(x[j], p, c);
        dx = G[j] * p * c;
      }
      dx += add[e];
    } else {
      if (dense) dx = s[j] * (G[j] - dot);
      if (RENORM) dx += add[e];
    }
    store_logit(static_cast<T*>(a.dlogits) + t * E + e, dx);
  }
}

template <typename T, int V, bool SIGMOID, bool RENORM>
cudaError_t launch_fwd(const RouteArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + kWarps - 1) / kWarps);
  const size_t smem = a.groups > 1 ? sizeof(float) * kWarps * a.E : 0;
  route_kernel<T, V, SIGMOID, RENORM><<<grid, kWarps * 32, smem, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int V, bool SIGMOID, bool RENORM>
cudaError_t launch_bwd(const RouteBwdArgs& a, cudaStream_t stream) {
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + kWarps - 1) / kWarps);
  route_backward_kernel<T, V, SIGMOID, RENORM>
      <<<grid, kWarps * 32, sizeof(float) * kWarps * a.E, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int V>
cudaError_t by_mode(const RouteArgs& a, bool sigmoid, bool renorm, cudaStream_t s) {
  if (sigmoid) return renorm ? launch_fwd<T, V, true, true>(a, s) : launch_fwd<T, V, true, false>(a, s);
  return renorm ? launch_fwd<T, V, false, true>(a, s) : launch_fwd<T, V, false, false>(a, s);
}
template <typename T, int V>
cudaError_t by_mode(const RouteBwdArgs& a, bool sigmoid, bool renorm, cudaStream_t s) {
  if (sigmoid) return renorm ? launch_bwd<T, V, true, true>(a, s) : launch_bwd<T, V, true, false>(a, s);
  return renorm ? launch_bwd<T, V, false, true>(a, s) : launch_bwd<T, V, false, false>(a, s);
}

template <typename T, typename Args>
cudaError_t by_width(const Args& a, bool sigmoid, bool renorm, cudaStream_t s) {
  if (a.E <= 32) return by_mode<T, 1>(a, sigmoid, renorm, s);
  if (a.E <= 64) return by_mode<T, 2>(a, sigmoid, renorm, s);
  if (a.E <= 128) return by_mode<T, 4>(a, sigmoid, renorm, s);
  if (a.E <= 256) return by_mode<T, 8>(a, sigmoid, renorm, s);
  if (a.E <= 512) return by_mode<T, 16>(a, sigmoid, renorm, s);
  return by_mode<T, 32>(a, sigmoid, renorm, s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, bool f32, bool sigmoid, bool renorm, cudaStream_t stream) {
  return f32 ? by_width<float>(a, sigmoid, renorm, stream)
             : by_width<__nv_bfloat16>(a, sigmoid, renorm, stream);
}
cudaError_t launch_route_backward(const RouteBwdArgs& a, bool f32, bool sigmoid, bool renorm,
                                  cudaStream_t stream) {
  return f32 ? by_width<float>(a, sigmoid, renorm, stream)
             : by_width<__nv_bfloat16>(a, sigmoid, renorm, stream);
}

}  // namespace mgw
