// Combine: routed rows back to token order, weighted, and its backward pass.
//
//   out[t]          = residual[t] + sum_k w[t, k] y[row_of[t, k]]
//   dy[row_of[t,k]] = w[t, k] dout[t]
//   dw[t, k]        = <dout[t], y[row_of[t, k]]>
//
// A row belongs to one (token, slot) pair, so nothing is summed across threads in the forward
// direction or in dy, and dw is a fixed-order block sum: results do not vary between runs.
// Both directions are bound by HBM: every y row is read once (and every dy row written once).
// Sums are fp32 in slot order; out and dy are rounded once.
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr unsigned kAll = 0xffffffffu;

// VEC elements of a row: 16 bytes, or one element when H or a pointer rules that out.
template <typename T, int VEC>
struct Pack {
  T v[VEC];
};
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

template <typename T, int VEC>
__device__ __forceinline__ void load(const T* p, float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    f[0] = to_f(*p);
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    const T* v = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) f[i] = to_f(v[i]);
  }
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* p, const float (&f)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(f[0]);
  } else {
    uint4 u;
    T* v = reinterpret_cast<T*>(&u);
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[i] = from_f<T>(f[i]);
    *reinterpret_cast<uint4*>(p) = u;
  }
}

// The pair's row, or -1 for a dropped one; a row outside y is reported and counts as dropped.
__device__ __forceinline__ int row_at(const int32_t* row_of, long long i, int M, int* status) {
  int r = row_of[i];
  if (r < -1 || r >= M) {
    if (status != nullptr) atomicOr(status, kDevBadIndex);
    r = -1;
  }
  return r;
}

// grid: (tokens, column blocks)
template <typename T, int VEC>
__global__ void __launch_bounds__(256) combine_kernel(CombineArgs a) {
  const long long t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * VEC;
  if (c >= a.H) return;
  const T* y = static_cast<const T*>(a.y);
  float acc[VEC];
  if (a.residual != nullptr) {
    load<T, VEC>(static_cast<const T*>(a.residual) + t * a.H + c, acc);
  } else {
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  }
  for (int k = 0; k < a.top_k; ++k) {
    const int r = row_at(a.row_of, t * a.top_k + k, a.M, a.status);
    if (r < 0) continue;
    const float w = a.weights != nullptr ? a.weights[t * a.top_k + k] : 1.0f;
    float v[VEC];
    load<T, VEC>(y + static_cast<long long>(r) * a.H + c, v);
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = fmaf(w, v[i], acc[i]);
  }
  store<T, VEC>(static_cast<T*>(a.out) + t * a.H + c, acc);
}

// One CTA per token.
template <typename T, int VEC>
__global__ void __launch_bounds__(256) combine_backward_kernel(CombineBwdArgs a) {
  __shared__ float s_sum[8];
  const long long t = blockIdx.x;
  const T* y = static_cast<const T*>(a.y);
  const T* d = static_cast<const T*>(a.dout) + t * a.H;
  for (int k = 0; k < a.top_k; ++k) {
    const int r = row_at(a.row_of, t * a.top_k + k, a.M, a.status);
    float dot = 0.0f;
    if (r >= 0) {
      const float w = a.weights != nullptr ? a.weights[t * a.top_k + k] : 1.0f;
      for (int c = threadIdx.x * VEC; c < a.H; c += blockDim.x * VEC) {
        float g[VEC], v[VEC];
        load<T, VEC>(d + c, g);
        if (a.dweights != nullptr) {
          load<T, VEC>(y + static_cast<long long>(r) * a.H + c, v);
#pragma unroll
          for (int i = 0; i < VEC; ++i) dot = fmaf(g[i], v[i], dot);
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = w * g[i];
        store<T, VEC>(static_cast<T*>(a.dy) + static_cast<long long>(r) * a.H + c, v);
      }
    }
    if (a.dweights != nullptr) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(kAll, dot, s);
      if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float sum = 0.0f;
        for (unsigned w = 0; w < blockDim.x / 32; ++w) sum += s_sum[w];
        a.dweights[t * a.top_k + k] = r >= 0 ? sum : 0.0f;
      }
      __syncthreads();
    }
  }
}

bool vectors(int H, size_t el, const void* p0, const void* p1, const void* p2, const void* p3) {
  const uintptr_t bits = reinterpret_cast<uintptr_t>(p0) | reinterpret_cast<uintptr_t>(p1) |
                         reinterpret_cast<uintptr_t>(p2) | reinterpret_cast<uintptr_t>(p3);
  return (static_cast<size_t>(H) * el) % 16 == 0 && (bits & 15) == 0;
}

template <typename T, int VEC>
cudaError_t launch_fwd(const CombineArgs& a, cudaStream_t stream) {
  const int n = (a.H + VEC - 1) / VEC;
  const int threads = n >= 256 ? 256 : (n + 31) / 32 * 32;
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>((n + threads - 1) / threads));
  combine_kernel<T, VEC><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int VEC>
cudaError_t launch_bwd(const CombineBwdArgs& a, cudaStream_t stream) {
  const int n = (a.H + VEC - 1) / VEC;
  const int threads = n >= 256 ? 256 : (n + 31) / 32 * 32;
  combine_backward_kernel<T, VEC><<<static_cast<unsigned>(a.T), threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, bool f32, cudaStream_t stream) {
  const bool vec = vectors(a.H, f32 ? 4 : 2, a.y, a.residual, a.out, nullptr);
  if (f32) return vec ? launch_fwd<float, 4>(a, stream) : launch_fwd<float, 1>(a, stream);
  return vec ? launch_fwd<__nv_bfloat16, 8>(a, stream) : launch_fwd<__nv_bfloat16, 1>(a, stream);
}
cudaError_t launch_combine_backward(const CombineBwdArgs& a, bool f32, cudaStream_t stream) {
  const bool vec = vectors(a.H, f32 ? 4 : 2, a.y, a.dout, a.dy, nullptr);
  if (f32) return vec ? launch_bwd<float, 4>(a, stream) : launch_bwd<float, 1>(a, stream);
  return vec ? launch_bwd<__nv_bfloat16, 8>(a, stream) : launch_bwd<__nv_bfloat16, 1>(a, stream);
}

}  // namespace mgw
