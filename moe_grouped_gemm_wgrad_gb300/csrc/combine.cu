// Combine: routed rows back to token order, weighted, and its backward pass.
//
//   out[t]          = residual[t] + sum_k w[t, k] y[row_of[t, k]]
//   dy[row_of[t,k]] = w[t, k] dout[t]
//   dw[t, k]        = <dout[t], y[row_of[t, k]]>
//
// A row belongs to one (token, slot) pair, so nothing is summed across threads in the forward
// direction or in dy, and dw is a fixed-order block sum: results do not vary between runs.
// Sums are fp32 in slot order; out and dy are rounded once.
//
// Both directions are bound by HBM: every y row is read once (and every dy row written once).
// What it takes to reach it is loads in flight: a thread keeps one 16-byte piece of the token
// and asks for the pieces of eight slots before it uses the first (their rows and weights come
// from shared memory, read once per CTA).  Rows whose width is not a multiple of 16 bytes
// start between 16-byte boundaries: a thread then takes two to four narrower words of each row,
// a warp's width apart, so that a warp's loads stay contiguous.  8192 x 8 x 4096 bf16, a graph's
// replay less an empty one's 4 us: forward with residual 101 us (6.6 TB/s, the copy rate), backward
// 164 us (6.9 TB/s; part of y is still in L2).
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

constexpr int kSlots = 8;      // slots whose loads are in flight together
constexpr int kMaxThreads = 256;

// Rows and weights of a token's slots to shared memory; -1 for a dropped pair.  A row outside
// y is reported and counts as dropped.
__device__ __forceinline__ void load_slots(const int32_t* row_of, const float* weights, long long t,
                                           int top_k, int M, int* status, int* s_row, float* s_w) {
  if (threadIdx.x < static_cast<unsigned>(top_k)) {
    const long long i = t * top_k + threadIdx.x;
    int r = row_of[i];
    if (r < -1 || r >= M) {
      if (status != nullptr) atomicOr(status, kDevBadIndex);
      r = -1;
    }
    s_row[threadIdx.x] = r;
    s_w[threadIdx.x] = weights != nullptr ? weights[i] : 1.0f;
  }
  __syncthreads();
}

// Word of AB bytes.
template <int AB>
struct Word;
template <>
struct Word<16> { using type = uint4; };
template <>
struct Word<8> { using type = uint2; };
template <>
struct Word<4> { using type = uint32_t; };
template <>
struct Word<2> { using type = uint16_t; };

// A thread's elements of a row: one 16-byte word, or kWords narrower ones a warp's width apart.
template <typename T, int AB>
struct Piece {
  static constexpr int kWords = AB == 16 ? 1 : AB == 8 ? 2 : 4;
  static constexpr int kPer = AB / static_cast<int>(sizeof(T));  // elements of a word
  static constexpr int N = kWords * kPer;
  using W = typename Word<AB>::type;
  W raw[kWords];
  // first column of piece i, and its number for rows of H columns
  static __device__ __forceinline__ int first(int i) { return (i / 32) * 32 * N + (i % 32) * kPer; }
  static __host__ __device__ __forceinline__ int count(int H) {
    return AB == 16 ? H / N : (H + 32 * N - 1) / (32 * N) * 32;
  }
  __device__ __forceinline__ void load(const T* row, int c, int H) {
#pragma unroll
    for (int q = 0; q < kWords; ++q)
      if (AB == 16 || c + q * 32 * kPer < H)
        raw[q] = *reinterpret_cast<const W*>(row + c + q * 32 * kPer);
      else
        raw[q] = W{};
  }
  __device__ __forceinline__ float at(int j) const {
    return to_f(reinterpret_cast<const T*>(&raw[j / kPer])[j % kPer]);
  }
  static __device__ __forceinline__ void store(T* row, int c, int H, const float (&f)[N]) {
#pragma unroll
    for (int q = 0; q < kWords; ++q) {
      W w;
      T* v = reinterpret_cast<T*>(&w);
#pragma unroll
      for (int j = 0; j < kPer; ++j) v[j] = from_f<T>(f[q * kPer + j]);
      if (AB == 16 || c + q * 32 * kPer < H) *reinterpret_cast<W*>(row + c + q * 32 * kPer) = w;
    }
  }
};

// grid: (tokens, column blocks); a thread owns one piece of the token.
// Five CTAs of 256 threads per SM.  8192 x 8 x 4096 without a residual, events around a call with
// dirty lines of other data in L2: 107 us, with four CTAs 111, with six, where the eight pieces
// spill out of flight, 119; CTAs of 128 or 512 threads cost 18 and 9% more.
template <typename T, int AB>
__global__ void __launch_bounds__(kMaxThreads, 5) combine_kernel(CombineArgs a) {
  using P = Piece<T, AB>;
  __shared__ int s_row[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  const long long t = blockIdx.x;
  const int c = P::first(blockIdx.y * blockDim.x + threadIdx.x);
  const bool in = c < a.H;
  P res;
  if (a.residual != nullptr && in) res.load(static_cast<const T*>(a.residual) + t * a.H, c, a.H);
  load_slots(a.row_of, a.weights, t, a.top_k, a.M, a.status, s_row, s_w);
  if (!in) return;
  float acc[P::N];
#pragma unroll
  for (int j = 0; j < P::N; ++j) acc[j] = a.residual != nullptr ? res.at(j) : 0.0f;
  const T* y = static_cast<const T*>(a.y);
  for (int k0 = 0; k0 < a.top_k; k0 += kSlots) {
    P v[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      const int r = k0 + k < a.top_k ? s_row[k0 + k] : -1;
      if (r >= 0) v[k].load(y + static_cast<long long>(r) * a.H, c, a.H);
    }
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
      if (k0 + k < a.top_k && s_row[k0 + k] >= 0) {
        const float w = s_w[k0 + k];
#pragma unroll
        for (int j = 0; j < P::N; ++j) acc[j] = fmaf(w, v[k].at(j), acc[j]);
      }
    }
  }
  P::store(static_cast<T*>(a.out) + t * a.H, c, a.H, acc);
}

// One CTA per token.  Every thread keeps its partial of each of kSlots dot products; the block
// sums them together (warp shuffles, then one warp over the warps' sums).
template <typename T, int AB>
__global__ void __launch_bounds__(kMaxThreads) combine_backward_kernel(CombineBwdArgs a) {
  using P = Piece<T, AB>;
  __shared__ int s_row[kMaxTopK];
  __shared__ float s_w[kMaxTopK];
  __shared__ float s_sum[kMaxThreads / 32][kSlots];
  const long long t = blockIdx.x;
  load_slots(a.row_of, a.weights, t, a.top_k, a.M, a.status, s_row, s_w);
  const T* d = static_cast<const T*>(a.dout) + t * a.H;
  const T* y = static_cast<const T*>(a.y);
  T* dy = static_cast<T*>(a.dy);
  const int pieces = P::count(a.H);
  for (int k0 = 0; k0 < a.top_k; k0 += kSlots) {
    float dot[kSlots];
#pragma unroll
    for (int k = 0; k < kSlots; ++k) dot[k] = 0.0f;
    for (int i = threadIdx.x; i < pieces; i += blockDim.x) {
      const int c = P::first(i);
      P g;
      g.load(d, c, a.H);
      P v[kSlots];
      if (a.dweights != nullptr) {
#pragma unroll
        for (int k = 0; k < kSlots; ++k) {
          const int r = k0 + k < a.top_k ? s_row[k0 + k] : -1;
          if (r >= 0) v[k].load(y + static_cast<long long>(r) * a.H, c, a.H);
        }
      }
      float gf[P::N];
#pragma unroll
      for (int j = 0; j < P::N; ++j) gf[j] = g.at(j);
#pragma unroll
      for (int k = 0; k < kSlots; ++k) {
        const int r = k0 + k < a.top_k ? s_row[k0 + k] : -1;
        if (r < 0) continue;
        const float w = s_w[k0 + k];
        float o[P::N];
#pragma unroll
        for (int j = 0; j < P::N; ++j) {
          if (a.dweights != nullptr) dot[k] = fmaf(gf[j], v[k].at(j), dot[k]);
          o[j] = w * gf[j];
        }
        P::store(dy + static_cast<long long>(r) * a.H, c, a.H, o);
      }
    }
    if (a.dweights == nullptr) continue;
#pragma unroll
    for (int k = 0; k < kSlots; ++k) {
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) dot[k] += __shfl_xor_sync(kAll, dot[k], s);
    }
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int k = 0; k < kSlots; ++k) s_sum[threadIdx.x >> 5][k] = dot[k];
    }
    __syncthreads();
    const int k = k0 + static_cast<int>(threadIdx.x);
    if (threadIdx.x < kSlots && k < a.top_k) {
      float sum = 0.0f;
      for (unsigned w = 0; w < blockDim.x / 32; ++w) sum += s_sum[w][threadIdx.x];
      a.dweights[t * a.top_k + k] = s_row[k] >= 0 ? sum : 0.0f;
    }
    __syncthreads();
  }
}

// The widest word that rows of H elements of `el` bytes start at multiples of (the C ABI asks
// for 16-byte aligned matrices).
int word_bytes(int H, int el) {
  const long long row = static_cast<long long>(H) * el;
  return row % 16 == 0 ? 16 : row % 8 == 0 ? 8 : row % 4 == 0 ? 4 : 2;
}

int threads_for(int pieces) { return pieces >= kMaxThreads ? kMaxThreads : (pieces + 31) / 32 * 32; }

template <typename T, int AB>
cudaError_t launch_word(const CombineArgs& a, cudaStream_t stream) {
  const int n = Piece<T, AB>::count(a.H);
  const int threads = threads_for(n);
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>((n + threads - 1) / threads));
  combine_kernel<T, AB><<<grid, threads, 0, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int AB>
cudaError_t launch_word(const CombineBwdArgs& a, cudaStream_t stream) {
  const int n = Piece<T, AB>::count(a.H);
  combine_backward_kernel<T, AB>
      <<<static_cast<unsigned>(a.T), threads_for(n), 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename Args>
cudaError_t launch_type(const Args& a, bool f32, cudaStream_t stream) {
  const int word = word_bytes(a.H, f32 ? 4 : 2);
  if (f32)
    return word == 16  ? launch_word<float, 16>(a, stream)
           : word == 8 ? launch_word<float, 8>(a, stream)
                       : launch_word<float, 4>(a, stream);
  return word == 16  ? launch_word<__nv_bfloat16, 16>(a, stream)
         : word == 8 ? launch_word<__nv_bfloat16, 8>(a, stream)
         : word == 4 ? launch_word<__nv_bfloat16, 4>(a, stream)
                     : launch_word<__nv_bfloat16, 2>(a, stream);
}

}  // namespace

cudaError_t launch_combine(const CombineArgs& a, bool f32, cudaStream_t stream) {
  return launch_type(a, f32, stream);
}
cudaError_t launch_combine_backward(const CombineBwdArgs& a, bool f32, cudaStream_t stream) {
  return launch_type(a, f32, stream);
}

}  // namespace mgw
