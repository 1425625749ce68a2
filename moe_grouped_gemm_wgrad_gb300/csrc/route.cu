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
// L lanes of a warp per token, V experts a lane: lane l of the token holds experts l V ..
// l V + V - 1, so of equal values the lowest lane's is the lowest index.  Up to 256 experts
// take V = 8 (one or two 16-byte loads) and L = 4, 8, 16 or 32: eight, four, two or one token per
// warp, as few lanes as hold the experts, with up to two choices a lane (both ways, bf16 softmax:
// 65536 x 8 top 2 30 -> 22 us against eight lanes, 40000 x 64 top 12 40 -> 26 against sixteen).
// A lane sorts its eight keys once; each of the top_k rounds is then a maximum over the token's
// lanes, one ballot, and a shift of the winning lane's list.  Beyond 256 experts a lane keeps its
// 16 or 32 keys unsorted and looks through them when it wins.  bf16 logits without a bias fit
// one 32-bit key with their index below them: no ballot, no second list.  The renormalised
// softmax needs the chosen logits only; sums are fp32.
//
// The work is instruction issue and latency, not bytes.  65536 x 64 (softmax, top 8, graph
// replay with its launch): 30 us with a warp per token and two experts a lane, 17.5 with this
// layout, 15.5 with one-word keys; reading and writing it takes 2.
#include <cuda_bf16.h>

#include <cstdint>
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;  // per CTA
constexpr float kNegInf = -__builtin_huge_valf();

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// V consecutive elements by 16-byte pieces.
template <int V>
__device__ __forceinline__ void load_vec(const float* p, float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 4) {
    const float4 f = *reinterpret_cast<const float4*>(p + j);
    x[j] = f.x, x[j + 1] = f.y, x[j + 2] = f.z, x[j + 3] = f.w;
  }
}
template <int V>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p + j);
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __bfloat1622float2(h[i]);
      x[j + 2 * i] = f.x, x[j + 2 * i + 1] = f.y;
    }
  }
}
template <int V>
__device__ __forceinline__ void store_vec(float* p, const float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 4)
    *reinterpret_cast<float4*>(p + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
}
template <int V>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; j += 8) {
    uint4 u;
    __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[j + 2 * i], x[j + 2 * i + 1]);
    *reinterpret_cast<uint4*>(p + j) = u;
  }
}

// Order-preserving map of a float (not NaN) to an unsigned integer; both zeros map alike.
// 0 is below every float's key and stands for "not available".
__device__ __forceinline__ uint32_t key_of(float f) {
  const uint32_t u = __float_as_uint(f == 0.0f ? 0.0f : f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}

// Reductions over the token's L lanes.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v += __shfl_xor_sync(kAll, v, d);
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = L / 2; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, d));
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(kAll, v);
  } else {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) v = max(v, __shfl_xor_sync(kAll, v, d));
    return v;
  }
}
// The lowest of the token's lanes for which p holds, or -1.
template <int L>
__device__ __forceinline__ int lowest_lane(bool p, int lane) {
  unsigned b = __ballot_sync(kAll, p);
  if constexpr (L < 32) b &= ((1u << L) - 1u) << (lane & ~(L - 1));
  return __ffs(b) - 1;
}

// e^(x - m), exactly 1 at x == m (also when both are infinite)
__device__ __forceinline__ float exp_from(float x, float m) { return x == m ? 1.0f : expf(x - m); }

// The logistic function and its complement from e^-|x|, which cannot overflow.
__device__ __forceinline__ void logistic(float x, float& s, float& c) {
  const float q = expf(-fabsf(x));
  const float r = __fdividef(1.0f, 1.0f + q);  // 1 <= 1 + q <= 2
  s = x >= 0.0f ? r : q * r;
  c = x >= 0.0f ? q * r : r;
}

// The same with the score divided by e^base, for base = min(the best chosen logit, 0): scores that
// are only compared with each other (renormalised weights) then never all underflow.
__device__ __forceinline__ void logistic_from(float x, float base, float& s, float& c) {
  const float q = expf(-fabsf(x));
  const float r = __fdividef(1.0f, 1.0f + q);
  s = x >= 0.0f ? r : exp_from(x, base) * r;
  c = x >= 0.0f ? q * r : r;
}

// This lane's V elements of its token's row of E: by 16-byte pieces where E is a multiple of V,
// else one by one.  (Other rows through shared memory, read and written as one run: slower, 36
// instead of 28 us for 40000 x 61 both ways, the lanes' sectors being in L1 anyway.)
template <int V, int L>
struct Row {
  int E, first;  // first: the lane's first expert
  bool live, vec;

  template <typename T>
  __device__ __forceinline__ void load(const T* row, float none, float (&x)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = none;
    if (live && vec) {
      if (first < E) load_vec<V>(row + first, x);
    } else if (live) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (first + j < E) x[j] = load_logit(row + first + j);
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, const float (&x)[V]) const {
    if (live && vec) {
      if (first < E) store_vec<V>(row + first, x);
    } else if (live) {
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (first + j < E) store_logit(row + first + j, x[j]);
    }
  }
};

// NaN logits are reported and count as masked.
template <int V>
__device__ __forceinline__ void mask_nan(float (&x)[V], int* status) {
  bool nan = false;
#pragma unroll
  for (int j = 0; j < V; ++j) nan |= x[j] != x[j];
  if (nan) {
#pragma unroll
    for (int j = 0; j < V; ++j)
      if (x[j] != x[j]) x[j] = kNegInf;
    if (status != nullptr) atomicOr(status, kDevBadLogit);
  }
}

// Scores of the row: softmax over the token's lanes (max and 1 / sum come back too), or the
// logistic function of each.
template <int V, int L, bool SIGMOID>
__device__ __forceinline__ void row_scores(const float (&x)[V], float (&s)[V], float& m, float& inv) {
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float c;
      logistic(x[j], s[j], c);
    }
  } else {
    m = x[0];
#pragma unroll
    for (int j = 1; j < V; ++j) m = fmaxf(m, x[j]);
    m = lanes_max<L>(m);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = x[j] == kNegInf ? 0.0f : exp_from(x[j], m);
      sum += s[j];
    }
    sum = lanes_sum<L>(sum);
    inv = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) s[j] *= inv;
  }
}

// Descending order of the lane's keys, equal ones in index order (a Batcher network for V = 8).
template <int V>
__device__ __forceinline__ void sort_keys(uint32_t (&key)[V], int (&idx)[V]) {
  auto swap = [&](int a, int b) {
    // a stays in front of an equal b unless b's index is lower
    const bool s = key[b] > key[a] || (key[b] == key[a] && idx[b] < idx[a]);
    const uint32_t k = key[a];
    const int i = idx[a];
    key[a] = s ? key[b] : k;
    idx[a] = s ? idx[b] : i;
    key[b] = s ? k : key[b];
    idx[b] = s ? i : idx[b];
  };
  static_assert(V == 8, "the network below is for eight keys");
  swap(0, 1), swap(2, 3), swap(4, 5), swap(6, 7);
  swap(0, 2), swap(1, 3), swap(4, 6), swap(5, 7);
  swap(1, 2), swap(5, 6);
  swap(0, 4), swap(1, 5), swap(2, 6), swap(3, 7);
  swap(2, 4), swap(3, 5);
  swap(1, 2), swap(3, 4), swap(5, 6);
}

// The same network for keys that differ, each carrying its index.
__device__ __forceinline__ void sort_packed(uint32_t (&key)[8]) {
  auto swap = [&](int a, int b) {
    const uint32_t hi = max(key[a], key[b]), lo = min(key[a], key[b]);
    key[a] = hi;
    key[b] = lo;
  };
  swap(0, 1), swap(2, 3), swap(4, 5), swap(6, 7);
  swap(0, 2), swap(1, 3), swap(4, 6), swap(5, 7);
  swap(1, 2), swap(5, 6);
  swap(0, 4), swap(1, 5), swap(2, 6), swap(3, 7);
  swap(2, 4), swap(3, 5);
  swap(1, 2), swap(3, 4), swap(5, 6);
}

// Choices that a lane keeps: lane l of the token has the l-th, and with fewer than 32 lanes to a
// token the (L + l)-th.
template <int L>
constexpr int kChoices = L < 32 ? 2 : 1;

// The token's top_k best of keys that each hold a 16-bit value above 65535 - its index.
template <int V, int L>
__device__ __forceinline__ void pick_packed(uint32_t (&key)[V], int top_k, int sub, int (&my_e)[kChoices<L>]) {
  if constexpr (V == 8) sort_packed(key);
  uint32_t head = key[0];
  if constexpr (V != 8) {
#pragma unroll
    for (int j = 1; j < V; ++j) head = max(head, key[j]);
  }
  auto round = [&](int k, int& mine) {
    const uint32_t best = lanes_max<L>(head);
    if (sub == k && best != 0u) mine = 65535 - static_cast<int>(best & 65535u);
    const bool won = head == best;
    if constexpr (V == 8) {
#pragma unroll
      for (int j = 0; j + 1 < V; ++j) key[j] = won ? key[j + 1] : key[j];
      key[V - 1] = won ? 0u : key[V - 1];
      head = key[0];
    } else if (won) {
      head = 0u;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (key[j] == best) key[j] = 0u;
        head = max(head, key[j]);
      }
    }
  };
#pragma unroll
  for (int r = 0; r < kChoices<L>; ++r)
    for (int k = 0; k < min(top_k - r * L, L); ++k) round(k, my_e[r]);
}

template <typename T, int V, int L, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kWarps * 32) route_kernel(RouteArgs a) {
  extern __shared__ float s_vals[];  // groups that are not whole lanes: 32 V values per warp
  const int lane = static_cast<int>(lane_id());
  const int sub = lane % L;  // lane of the token
  const long long t = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * (32 / L) + lane / L;
  const bool live = t < a.T;
  const int E = a.E;
  const int first = sub * V;  // this lane's first expert
  const Row<V, L> at{E, first, live, E % V == 0};
  const T* row = static_cast<const T*>(a.logits) + t * E;
  float x[V], s[V], m = 0.0f, inv = 0.0f;
  at.load(row, kNegInf, x);
  mask_nan(x, a.status);
  const bool need_scores = (SIGMOID ? a.bias != nullptr : !RENORM || a.bias != nullptr) ||
                           a.scores != nullptr || (a.groups > 1 && a.group_best == 2);
  if (need_scores) row_scores<V, L, SIGMOID>(x, s, m, inv);
  if (a.scores != nullptr) at.store(a.scores + t * E, s);
  uint32_t key[V];
  if (a.bias != nullptr) {
    float b[V];
    Row<V, L>{E, first, true, at.vec}.load(a.bias, 0.0f, b);
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = x[j] == kNegInf ? 0u : key_of(s[j] + b[j]);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) key[j] = x[j] == kNegInf ? 0u : key_of(x[j]);
  }
  if (a.groups > 1) {
    const int per = E / a.groups;
    const bool sum2 = a.group_best == 2;
    const int lanes = per / V;  // lanes of a group, when groups are whole runs of 2^i lanes
    if (per % V == 0 && (lanes & (lanes - 1)) == 0) {
      float b1 = kNegInf, b2 = kNegInf;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float v = key[j] == 0u ? kNegInf : (sum2 && a.bias == nullptr ? s[j] : value_of(key[j]));
        b2 = fmaxf(b2, fminf(b1, v));
        b1 = fmaxf(b1, v);
      }
      for (int d = lanes / 2; d > 0; d >>= 1) {
        const float o1 = __shfl_xor_sync(kAll, b1, d), o2 = __shfl_xor_sync(kAll, b2, d);
        b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
        b1 = fmaxf(b1, o1);
      }
      uint32_t gkey = b1 == kNegInf ? 0u : key_of(sum2 && b2 != kNegInf ? b1 + b2 : b1);
      bool kept = false;
      for (int i = 0; i < a.top_groups; ++i) {
        const uint32_t best = lanes_max<L>(gkey);
        const int src = lowest_lane<L>(gkey == best && best != 0u, lane);
        if (src >= 0 && (lane ^ src) < lanes) {  // same run of lanes: only low bits differ
          kept = true;
          gkey = 0u;
        }
      }
      if (!kept) {
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = 0u;
      }
    } else {
      // group values through shared memory: the token's lane g takes groups g, g + L, ..
      float* vals = s_vals + (threadIdx.x >> 5) * (32 * V) + lane / L * E;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (first + j < E)
          vals[first + j] =
              key[j] == 0u ? kNegInf : (sum2 && a.bias == nullptr ? s[j] : value_of(key[j]));
      __syncwarp();
      constexpr int kMine = 32 / L;  // groups of a lane, at most
      uint32_t gkey[kMine];
#pragma unroll
      for (int q = 0; q < kMine; ++q) {
        const int g = sub + q * L;
        float b1 = kNegInf, b2 = kNegInf;
        if (g < a.groups) {
          for (int i = 0; i < per; ++i) {
            const float v = vals[g * per + i];
            b2 = fmaxf(b2, fminf(b1, v));
            b1 = fmaxf(b1, v);
          }
        }
        gkey[q] = b1 == kNegInf ? 0u : key_of(sum2 && b2 != kNegInf ? b1 + b2 : b1);
      }
      unsigned kept = 0;
      for (int i = 0; i < a.top_groups; ++i) {
        uint32_t mine = gkey[0];
#pragma unroll
        for (int q = 1; q < kMine; ++q) mine = max(mine, gkey[q]);
        const uint32_t best = lanes_max<L>(mine);
        // the lowest group of that value: the largest 32 - g
        uint32_t c = 0;
#pragma unroll
        for (int q = 0; q < kMine; ++q)
          if (best != 0u && gkey[q] == best) c = max(c, static_cast<uint32_t>(32 - (sub + q * L)));
        c = lanes_max<L>(c);
        if (c != 0u) {
          const int g = 32 - static_cast<int>(c);
          kept |= 1u << g;
#pragma unroll
          for (int q = 0; q < kMine; ++q)
            if (g == sub + q * L) gkey[q] = 0u;
        }
      }
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (first + j < E && !((kept >> ((first + j) / per)) & 1u)) key[j] = 0u;
    }
  }
  constexpr int R = kChoices<L>;
  int my_e[R];
#pragma unroll
  for (int r = 0; r < R; ++r) my_e[r] = -1;
  if (std::is_same<T, __nv_bfloat16>::value && a.bias == nullptr) {
    // a bf16 value is the upper half of its fp32 key
#pragma unroll
    for (int j = 0; j < V; ++j)
      key[j] = key[j] == 0u ? 0u : (key[j] & 0xffff0000u) | static_cast<uint32_t>(65535 - (first + j));
    pick_packed<V, L>(key, a.top_k, sub, my_e);
  } else if constexpr (V == 8) {
    int idx[V];
#pragma unroll
    for (int j = 0; j < V; ++j) idx[j] = j;
    sort_keys<V>(key, idx);
    auto round = [&](int k, int& mine) {
      const uint32_t best = lanes_max<L>(key[0]);
      const int src = lowest_lane<L>(key[0] == best && best != 0u, lane);
      const int e = __shfl_sync(kAll, first + idx[0], src < 0 ? lane : src);
      if (sub == k && src >= 0) mine = e;
      if (lane == src) {
#pragma unroll
        for (int j = 0; j + 1 < V; ++j) key[j] = key[j + 1], idx[j] = idx[j + 1];
        key[V - 1] = 0u;
      }
    };
#pragma unroll
    for (int r = 0; r < R; ++r)
      for (int k = 0; k < min(a.top_k - r * L, L); ++k) round(k, my_e[r]);
  } else {
    uint32_t head = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) head = max(head, key[j]);
    for (int k = 0; k < a.top_k; ++k) {
      const uint32_t best = lanes_max<L>(head);
      if (best == 0u) break;
      const int src = lowest_lane<L>(head == best, lane);
      int pick = 0;
      if (lane == src) {
        bool found = false;
        head = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if (!found && key[j] == best) {
            found = true;
            pick = j;
            key[j] = 0u;
          }
          head = max(head, key[j]);
        }
      }
      pick = __shfl_sync(kAll, first + pick, src);
      if (lane == k) my_e[0] = pick;
    }
  }
  // weights of the chosen, from their logits
  const bool more = R > 1 && a.top_k > L;  // a lane's second choice counts
  float w[R], xk[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    w[r] = 0.0f;
    xk[r] = my_e[r] >= 0 ? load_logit(row + my_e[r]) : kNegInf;
  }
  float top = kNegInf;
  if constexpr (RENORM) top = lanes_max<L>(R > 1 ? fmaxf(xk[0], xk[R - 1]) : xk[0]);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if ((r > 0 && !more) || my_e[r] < 0) continue;
    float c;
    if constexpr (SIGMOID && RENORM)
      logistic_from(xk[r], fminf(top, 0.0f), w[r], c);
    else if constexpr (SIGMOID)
      logistic(xk[r], w[r], c);
    else if constexpr (RENORM)
      w[r] = exp_from(xk[r], top);
    else
      w[r] = exp_from(xk[r], m) * inv;
  }
  if constexpr (RENORM) {
    const float sum = lanes_sum<L>(R > 1 ? w[0] + w[R - 1] : w[0]);
#pragma unroll
    for (int r = 0; r < R; ++r) w[r] = sum > 0.0f ? w[r] / sum : 0.0f;
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (live && sub + r * L < a.top_k) {
      a.expert_idx[t * a.top_k + sub + r * L] = my_e[r];
      a.weights[t * a.top_k + sub + r * L] = w[r] * a.scale;
    }
  }
}

// dlogits, with the forward kernel's lanes.  With G = dL/ds (the scores' own gradient plus the
// weights'): softmax dx = s (G - sum s G), logistic dx = G s (1 - s).  Renormalised weights
// w = scale * p depend on the chosen only: their part is p_k (g_k - sum_j p_j g_j), g = scale *
// dw, times (1 - s_k) for the logistic function.  The chosen experts' terms reach the lanes
// that own them through shared memory.
template <typename T, int V, int L, bool SIGMOID, bool RENORM>
__global__ void __launch_bounds__(kWarps * 32) route_backward_kernel(RouteBwdArgs a) {
  __shared__ __align__(16) float s_add[kWarps][32 * V];
  const int lane = static_cast<int>(lane_id());
  const int sub = lane % L;
  const int warp = threadIdx.x >> 5;
  const long long t = (static_cast<long long>(blockIdx.x) * kWarps + warp) * (32 / L) + lane / L;
  const bool live = t < a.T;
  const int E = a.E;
  const Row<V, L> at{E, sub * V, live, E % V == 0};
  const T* row = static_cast<const T*>(a.logits) + t * E;
  // the chosen experts first: their logits' addresses depend on them
  constexpr int R = kChoices<L>;
  int e[R];
  float g[R], xk[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    e[r] = -1, g[r] = 0.0f, xk[r] = kNegInf;
    if (a.dweights != nullptr && live && sub + r * L < a.top_k) {
      e[r] = a.expert_idx[t * a.top_k + sub + r * L];
      g[r] = a.dweights[t * a.top_k + sub + r * L] * a.scale;
    }
  }
  float x[V], s[V], add[V], G[V], m = 0.0f, inv = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) add[j] = G[j] = s[j] = 0.0f;
  at.load(row, kNegInf, x);
  mask_nan(x, a.status);
  if (a.dscores != nullptr) at.load(a.dscores + t * E, 0.0f, G);
  const bool dense = !SIGMOID && (!RENORM || a.dscores != nullptr);
  // the chosen experts' terms: added to G (plain softmax) or straight to dx (the others)
  if (a.dweights != nullptr) {
    const bool more = R > 1 && a.top_k > L;
    float term[R], p[R], c[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (e[r] < -1 || e[r] >= E) {
        if (a.status != nullptr) atomicOr(a.status, kDevBadIndex);
        e[r] = -1;
      }
      if (e[r] >= 0) xk[r] = load_logit(row + e[r]);
      if (!(xk[r] > kNegInf)) e[r] = -1, g[r] = 0.0f, xk[r] = kNegInf;  // no expert, masked, or not a number
      p[r] = 0.0f, c[r] = 1.0f;
    }
    float top = kNegInf;
    if constexpr (RENORM) top = lanes_max<L>(R > 1 ? fmaxf(xk[0], xk[R - 1]) : xk[0]);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      term[r] = g[r];
      if ((r > 0 && !more) || e[r] < 0) continue;
      if constexpr (SIGMOID && RENORM)
        logistic_from(xk[r], fminf(top, 0.0f), p[r], c[r]);
      else if constexpr (SIGMOID)
        logistic(xk[r], p[r], c[r]);
      else if constexpr (RENORM)
        p[r] = exp_from(xk[r], top);
      if constexpr (SIGMOID && !RENORM) term[r] = g[r] * p[r] * c[r];
    }
    if constexpr (RENORM) {
      const float sum = lanes_sum<L>(R > 1 ? p[0] + p[R - 1] : p[0]);
#pragma unroll
      for (int r = 0; r < R; ++r) p[r] = sum > 0.0f ? p[r] / sum : 0.0f;
      const float dot = lanes_sum<L>(R > 1 ? p[0] * g[0] + p[R - 1] * g[R - 1] : p[0] * g[0]);
#pragma unroll
      for (int r = 0; r < R; ++r) term[r] = p[r] * (g[r] - dot) * c[r];
    }
    float* mine = s_add[warp] + lane * V;
#pragma unroll
    for (int j = 0; j < V; j += 4) *reinterpret_cast<float4*>(mine + j) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    __syncwarp();
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (e[r] >= 0) s_add[warp][(lane - sub) * V + e[r]] = term[r];  // a token's experts differ
    __syncwarp();
    load_vec<V>(mine, add);
  }
  float dx[V];
  if constexpr (SIGMOID) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float p = 0.0f, c = 0.0f;
      if (a.dscores != nullptr && x[j] != kNegInf) logistic(x[j], p, c);
      dx[j] = (x[j] != kNegInf ? G[j] * p * c : 0.0f) + add[j];
    }
  } else {
    float dot = 0.0f;
    if (dense) {
      row_scores<V, L, false>(x, s, m, inv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        if (x[j] == kNegInf) G[j] = 0.0f;
        if (!RENORM) G[j] += add[j];
        dot += s[j] * G[j];
      }
      dot = lanes_sum<L>(dot);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dx[j] = s[j] * (G[j] - dot);
      if (RENORM) dx[j] += add[j];
      if (x[j] == kNegInf) dx[j] = 0.0f;  // whatever dot is
    }
  }
  at.store(static_cast<T*>(a.dlogits) + t * E, dx);
}

template <typename T, int V, int L, bool SIGMOID, bool RENORM>
cudaError_t launch_one(const RouteArgs& a, cudaStream_t stream) {
  constexpr int kTokens = kWarps * (32 / L);  // per CTA
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + kTokens - 1) / kTokens);
  const size_t smem = a.groups > 1 ? sizeof(float) * kWarps * 32 * V : 0;
  route_kernel<T, V, L, SIGMOID, RENORM><<<grid, kWarps * 32, smem, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int V, int L, bool SIGMOID, bool RENORM>
cudaError_t launch_one(const RouteBwdArgs& a, cudaStream_t stream) {
  constexpr int kTokens = kWarps * (32 / L);
  const unsigned grid = static_cast<unsigned>((static_cast<long long>(a.T) + kTokens - 1) / kTokens);
  route_backward_kernel<T, V, L, SIGMOID, RENORM><<<grid, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int V, int L, typename Args>
cudaError_t by_mode(const Args& a, bool sigmoid, bool renorm, cudaStream_t s) {
  if (sigmoid) return renorm ? launch_one<T, V, L, true, true>(a, s) : launch_one<T, V, L, true, false>(a, s);
  return renorm ? launch_one<T, V, L, false, true>(a, s) : launch_one<T, V, L, false, false>(a, s);
}

template <typename T, typename Args>
cudaError_t by_width(const Args& a, bool sigmoid, bool renorm, cudaStream_t s) {
  if (a.E <= 32 && a.top_k <= 8) return by_mode<T, 8, 4>(a, sigmoid, renorm, s);
  if (a.E <= 64 && a.top_k <= 16) return by_mode<T, 8, 8>(a, sigmoid, renorm, s);
  if (a.E <= 128) return by_mode<T, 8, 16>(a, sigmoid, renorm, s);
  if (a.E <= 256) return by_mode<T, 8, 32>(a, sigmoid, renorm, s);
  if (a.E <= 512) return by_mode<T, 16, 32>(a, sigmoid, renorm, s);
  return by_mode<T, 32, 32>(a, sigmoid, renorm, s);
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
