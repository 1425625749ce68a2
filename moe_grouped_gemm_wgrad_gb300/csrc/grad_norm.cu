// The norm of all gradients of a model together, and the gradients scaled down to a largest norm:
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + eps))
//
// HBM bounds both.  The tensors' table (address, size, type of each) rides in the kernel's
// parameters, up to 32 KB of them: nothing is copied to the device and a captured call replays as it
// is.  Every tensor is cut into chunks of 32 KB, and every CTA takes a run of the chunks of all tensors
// that is equally long for all CTAs, so large and tiny tensors mix without a tail.
//
// Squares are summed in fp32 over one thread's share of a chunk (at most 64 elements, in eight
// sums), these are added without loss (a pair of fp32 numbers, each addition's rounding error kept) and
// meet in fp64.  A share whose sum overflows, or is too small to be right (below 2^-80), is summed again
// in fp64: the norm is right wherever it is itself an fp32 number.
//
// Doubles are scarce here: FP64 runs two lanes an SM quarter, so only one warp of a CTA adds any (see
// block_sum), and the loads of whole chunks have no bounds checks, a pair of values is one packed
// multiply-add, what finding a chunk costs is shared by 32 KB.  64 x 1536 x 4096 bf16 (805 MB): norm 136
// us, 5.9 TB/s with what the launch before left to be written back (reading alone 7.1), clipping
// 247 us, 6.5 TB/s read and written.
//
// Up to kSmallChunks chunks one cluster of eight CTAs does it all, whose sums meet in shared memory: one
// launch instead of two (a launch costs the caller more than the bytes do).
//
// The clipping launch adds the CTAs' sums up in every CTA (a few KB, always in the same order) rather
// than wait for a launch in between; it walks the chunks backwards, so that what the norm read last is
// still in L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 32768;                // bytes
constexpr int kVecs = kChunk / 16 / kThreads;  // 16-byte pieces a thread has of a chunk
constexpr int kCtasPerSm = 4;
constexpr int kSmallTable = 128, kLargeTable = 1024;  // tensors of a launch
constexpr int kMostSms = 160;  // that a launch is sized for
constexpr int kSmallCluster = 8, kSmallThreads = 1024, kSmallChunks = 64;

struct Entry {
  const void* g;
  void* out;  // null: the norm only
  int64_t n;  // elements
};
// The tensors of one launch.  first[i]: chunks before tensor i; f32 as bits.
template <int CAP>
struct Table {
  Entry t[CAP];
  int first[CAP + 1];
  uint32_t f32[(CAP + 31) / 32];
  int count;
  double* sums;        // one per CTA of every launch
  int sums_at, total;  // this launch's first one; how many there are in all
  float* norm;
  const float* norm_in;  // clip to this norm; null: to that of the sums
  float max_norm, eps;
  int clip;
};
static_assert(sizeof(Table<kLargeTable>) <= 32764, "kernel parameters");
static_assert(sizeof(Table<kSmallTable>) <= 4096, "kernel parameters");

// A chunk of a tensor: whole 16-byte pieces (of the input's alignment) and, in the tensor's first and
// last chunk, the elements before and behind them.
struct Piece {
  const uint8_t* g;
  uint8_t* out;
  int64_t lo, hi;      // bytes of the chunk's 16-byte pieces, from the first aligned address on
  int head, tail;      // elements before and behind (first and last chunk)
  int64_t tail_at;     // element
  int skip;            // bytes from g to the first aligned address
  bool f32;
};

template <int CAP>
__device__ __forceinline__ Piece piece_of(const Table<CAP>& a, int i, int chunk) {
  const Entry& e = a.t[i];
  Piece p;
  p.f32 = (a.f32[i >> 5] >> (i & 31)) & 1u;
  const int size = p.f32 ? 4 : 2;
  p.g = static_cast<const uint8_t*>(e.g);
  p.out = static_cast<uint8_t*>(e.out);
  const int64_t bytes = e.n * size;
  int64_t skip = (16 - (reinterpret_cast<uintptr_t>(e.g) & 15)) & 15;
  if (skip > bytes) skip = bytes;
  p.skip = static_cast<int>(skip);
  const int64_t whole = (bytes - skip) & ~int64_t(15);
  const int64_t k = chunk - a.first[i];
  p.lo = k * kChunk;
  p.hi = p.lo + kChunk < whole ? p.lo + kChunk : whole;
  p.head = k == 0 ? p.skip / size : 0;
  const bool last = chunk + 1 == a.first[i + 1];
  p.tail = last ? static_cast<int>((bytes - skip - whole) / size) : 0;
  p.tail_at = (skip + whole) / size;
  return p;
}

// The largest i with first[i] <= chunk (tensors without elements have no chunk).  The parameters are cold
// at a launch's start, each line a miss: tensors of one size are found at once.
template <int CAP>
__device__ __forceinline__ int locate(const Table<CAP>& a, int chunk) {
  const int guess = min(static_cast<int>(__fdividef(static_cast<float>(chunk), static_cast<float>(a.first[a.count])) *
                                         static_cast<float>(a.count)),
                        a.count - 1);
  if (a.first[guess] <= chunk && chunk < a.first[guess + 1]) return guess;
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.first[mid] <= chunk)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float2 bf16_pair(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float element(const Piece& p, int64_t i) {
  return p.f32 ? reinterpret_cast<const float*>(p.g)[i]
               : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p.g)[i]);
}

// A thread's share of the squares: hi + lo, exact but for lo's own rounding, and what fp32 cannot hold.
struct Share {
  float hi, lo;
  double rest;
  __device__ __forceinline__ void add(float s) {
    const float t = hi + s, z = t - hi;
    lo += (hi - (t - z)) + (s - z);
    hi = t;
  }
};

// The sum of a CTA's shares, in all lanes of its first warp; s holds WARPS.  A double addition takes a
// warp 16 cycles here (two FP64 lanes an SM half), so the warps add up pairs of fp32 numbers and one of
// them the rest: with doubles throughout, in every thread, a CTA of 1024 took 10 us for it.
template <int WARPS>
__device__ __forceinline__ double block_sum(Share v, double* s) {
  constexpr unsigned kAll = 0xffffffffu;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const float hi = __shfl_xor_sync(kAll, v.hi, d), lo = __shfl_xor_sync(kAll, v.lo, d);
    v.add(hi);
    v.lo += lo;
  }
  if (__any_sync(kAll, v.rest != 0.0)) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v.rest += __shfl_xor_sync(kAll, v.rest, d);
  }
  if ((threadIdx.x & 31) == 0)
    s[threadIdx.x >> 5] = static_cast<double>(v.hi) + static_cast<double>(v.lo) + v.rest;
  __syncthreads();
  double sum = 0.0;
  if (threadIdx.x < 32) {
    if (threadIdx.x < WARPS) sum = s[threadIdx.x];
#pragma unroll
    for (int d = WARPS / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(kAll, sum, d);
  }
  return sum;
}

// kThreads threads share a chunk; a thread's number among them:
__device__ __forceinline__ int self() { return static_cast<int>(threadIdx.x) % kThreads; }

// A thread's 16-byte pieces of a chunk, zeros where it has none.
__device__ __forceinline__ void load_pieces(const Piece& p, uint4 (&w)[kVecs]) {
  const uint4* v = reinterpret_cast<const uint4*>(p.g + p.skip + p.lo) + self();
  const int n = static_cast<int>(p.hi - p.lo) >> 4;
  if (n == kChunk / 16) {
#pragma unroll
    for (int k = 0; k < kVecs; ++k) w[k] = v[k * kThreads];
  } else {
#pragma unroll
    for (int k = 0; k < kVecs; ++k)
      w[k] = self() + k * kThreads < n ? v[k * kThreads] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// s += (a a, b b) on a pair of fp32 numbers.
__device__ __forceinline__ void add_squares(uint64_t& s, uint32_t a, uint32_t b) {
  asm("{\n\t.reg .b64 v;\n\tmov.b64 v, {%1, %2};\n\tfma.rn.f32x2 %0, v, v, %0;\n\t}" : "+l"(s) : "r"(a), "r"(b));
}
__device__ __forceinline__ float both(uint64_t s) {
  return __uint_as_float(static_cast<uint32_t>(s)) + __uint_as_float(static_cast<uint32_t>(s >> 32));
}

// The squares' sum of a thread's pieces.
template <bool F32>
__device__ __forceinline__ float sum_squares(const uint4 (&w)[kVecs]) {
  uint64_t s[4] = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    if constexpr (F32) {
      add_squares(s[2 * (k & 1)], w[k].x, w[k].y);
      add_squares(s[2 * (k & 1) + 1], w[k].z, w[k].w);
    } else {
      add_squares(s[0], w[k].x << 16, w[k].x & 0xffff0000u);
      add_squares(s[1], w[k].y << 16, w[k].y & 0xffff0000u);
      add_squares(s[2], w[k].z << 16, w[k].z & 0xffff0000u);
      add_squares(s[3], w[k].w << 16, w[k].w & 0xffff0000u);
    }
  }
  return (both(s[0]) + both(s[1])) + (both(s[2]) + both(s[3]));
}
// (Reads the n pieces again rather than keep them in memory that a rare call could address.)
__device__ __noinline__ double sum_squares_wide(const uint4* v, int n, bool f32) {
  double d = 0.0;
  for (int i = self(); i < n; i += kThreads) {
    const uint4 w = v[i];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (f32) {
        const double f = __uint_as_float(u[j]);
        d += f * f;
      } else {
        const float2 f = bf16_pair(u[j]);
        d += static_cast<double>(f.x) * f.x + static_cast<double>(f.y) * f.y;
      }
    }
  }
  return d;
}

// The squares' sum over chunks c0, c0 + step, .. below c1, this thread's share.
template <int CAP>
__device__ __forceinline__ Share sum_chunks(const Table<CAP>& a, int c0, int c1, int step) {
  Share v = {0.0f, 0.0f, 0.0};
  int i = c0 < c1 ? locate(a, c0) : 0;
  for (int c = c0; c < c1; c += step) {
    while (c >= a.first[i + 1]) ++i;
    const Piece p = piece_of(a, i, c);
    uint4 w[kVecs];
    load_pieces(p, w);
    const float s = p.f32 ? sum_squares<true>(w) : sum_squares<false>(w);
    if (s < 0x1p120f && s >= 0x1p-80f) {
      v.add(s);
      if (v.hi >= 0x1p120f) v.rest += v.hi, v.hi = 0.0f;
    } else {
      uint32_t any = 0u;  // zeros all, as the gradients of parameters that a step did not reach
#pragma unroll
      for (int k = 0; k < kVecs; ++k) any |= w[k].x | w[k].y | w[k].z | w[k].w;
      if (any != 0u)
        v.rest += sum_squares_wide(reinterpret_cast<const uint4*>(p.g + p.skip + p.lo),
                                   static_cast<int>(p.hi - p.lo) >> 4, p.f32);
    }
    const int t = self();
    if (t < p.head + p.tail) {  // at most seven elements each
      const double f = element(p, t < p.head ? t : p.tail_at + (t - p.head));
      v.rest += f * f;
    }
  }
  return v;
}

// min(1, max_norm / (norm + eps)), but not for a norm that is not a number: then every gradient is none.
// Where the quotient would be none for numbers: an infinite norm gives 0 whatever max_norm, max_norm = 0
// gives 0 whatever the norm, and an infinite max_norm limits nothing.
__device__ __forceinline__ float clip_factor(float max_norm, float norm, float eps) {
  if (norm == INFINITY || (max_norm == 0.0f && norm == norm)) return 0.0f;
  if (max_norm == INFINITY && norm == norm) return 1.0f;
  const float f = max_norm / (norm + eps);
  return f > 1.0f ? 1.0f : f;
}

// Scales a chunk, whose pieces are in w.
__device__ __forceinline__ void scale_chunk(const Piece& p, const uint4 (&w)[kVecs], float f) {
  if (f == 1.0f && p.out == p.g) return;  // times 1, in place
  // the output's 16-byte pieces lie as the input's do, or they are stored element by element
  const bool same = ((reinterpret_cast<uintptr_t>(p.out) ^ reinterpret_cast<uintptr_t>(p.g)) & 15) == 0;
  const int n = static_cast<int>(p.hi - p.lo) >> 4;
#pragma unroll
  for (int k = 0; k < kVecs; ++k) {
    const int at = self() + k * kThreads;
    if (at >= n) continue;
    uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (p.f32) {
        u[j] = __float_as_uint(__uint_as_float(u[j]) * f);
      } else {
        const float2 x = bf16_pair(u[j]);
        const __nv_bfloat162 y = __floats2bfloat162_rn(x.x * f, x.y * f);
        u[j] = *reinterpret_cast<const uint32_t*>(&y);
      }
    }
    uint8_t* to = p.out + p.skip + p.lo + at * 16;
    if (same) {
      *reinterpret_cast<uint4*>(to) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (p.f32) {
          reinterpret_cast<uint32_t*>(to)[j] = u[j];
        } else {
          reinterpret_cast<uint16_t*>(to)[2 * j] = static_cast<uint16_t>(u[j]);
          reinterpret_cast<uint16_t*>(to)[2 * j + 1] = static_cast<uint16_t>(u[j] >> 16);
        }
      }
    }
  }
  const int t = self();
  if (t < p.head + p.tail) {
    const int64_t at = t < p.head ? t : p.tail_at + (t - p.head);
    const float x = element(p, at) * f;
    if (p.f32)
      reinterpret_cast<float*>(p.out)[at] = x;
    else
      reinterpret_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(x);
  }
}

// The launch before in the stream has ended and its results are there.  All launches here are programmatic
// dependents, the first of a call too: one after the other they take their own time and 0.6 us each, where
// plain launches of a few us start at multiples of 2.05 us (6 us: 6.6 against 8.2).  Every thread waits
// before it ends, so that a launch that has ended has none before it still running.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_norm_kernel(const __grid_constant__ Table<CAP> a) {
  __shared__ double s_sum[kWarps];
  const int chunks = a.first[a.count];
  const int c0 = static_cast<int>(static_cast<long long>(chunks) * blockIdx.x / gridDim.x);
  const int c1 = static_cast<int>(static_cast<long long>(chunks) * (blockIdx.x + 1) / gridDim.x);
  wait_for_launch_before();
  const double sum = block_sum<kWarps>(sum_chunks(a, c0, c1, 1), s_sum);
  if (threadIdx.x == 0) a.sums[a.sums_at + blockIdx.x] = sum;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// norm from all CTAs' sums, the same in every CTA; s_norm: one number.
__device__ __forceinline__ float total_norm(const double* sums, int total, float* s_norm) {
  if (threadIdx.x < 32) {
    double v = 0.0;
#pragma unroll 4
    for (int i = threadIdx.x; i < total; i += 32) v += sums[i];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
    if (threadIdx.x == 0) *s_norm = static_cast<float>(sqrt(v));
  }
  __syncthreads();
  return *s_norm;
}

__global__ void __launch_bounds__(32) grad_norm_end_kernel(const double* sums, int total, float* norm) {
  __shared__ float s_norm;
  wait_for_launch_before();
  const float n = total_norm(sums, total, &s_norm);
  if (threadIdx.x == 0) *norm = n;
}

template <int CAP>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) grad_clip_kernel(const __grid_constant__ Table<CAP> a) {
  __shared__ float s_norm;
  const int chunks = a.first[a.count];
  const int c0 = static_cast<int>(static_cast<long long>(chunks) * blockIdx.x / gridDim.x);
  const int c1 = static_cast<int>(static_cast<long long>(chunks) * (blockIdx.x + 1) / gridDim.x);
  int i = 0;
  Piece p = {};
  uint4 w[kVecs];
  auto load = [&](int c) {
    while (c < a.first[i]) --i;
    p = piece_of(a, i, c);
    load_pieces(p, w);
  };
  if (c0 < c1) i = locate(a, c1 - 1);
  // The launch before is the norm's: the gradients were there before it.  With a norm that the caller
  // knows it may be the gradients' own.
  const bool early = a.norm_in == nullptr && c0 < c1;
  if (early) load(c1 - 1);
  wait_for_launch_before();
  const float norm = a.norm_in != nullptr ? *a.norm_in : total_norm(a.sums, a.total, &s_norm);
  if (a.norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = norm;
  const float f = clip_factor(a.max_norm, norm, a.eps);
  for (int c = c1 - 1; c >= c0; --c) {
    if (!early || c != c1 - 1) load(c);
    scale_chunk(p, w, f);
  }
}

// Norm, or norm and clipping, of few chunks by one cluster, kThreads threads to a chunk.
template <int CAP>
__global__ void __launch_bounds__(kSmallThreads, 1) grad_small_kernel(const __grid_constant__ Table<CAP> a) {
  __shared__ double s_sum[kSmallThreads / 32];
  __shared__ double s_all[kSmallCluster];
  __shared__ float s_norm;
  constexpr int kGroups = kSmallThreads / kThreads * kSmallCluster;
  const int rank = static_cast<int>(cluster_ctarank());
  const int first = rank + kSmallCluster * static_cast<int>(threadIdx.x / kThreads);
  const int chunks = a.first[a.count];
  wait_for_launch_before();
  const double sum = block_sum<kSmallThreads / 32>(sum_chunks(a, first, chunks, kGroups), s_sum);
  cluster_sync();  // every CTA runs: its shared memory may be written
  if (threadIdx.x < kSmallCluster)
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(map_to_cta(smem_u32(&s_all[rank]), threadIdx.x)), "d"(sum)
                 : "memory");
  cluster_sync();
  if (threadIdx.x == 0) {
    double total = 0.0;
#pragma unroll
    for (int p = 0; p < kSmallCluster; ++p) total += s_all[p];
    s_norm = static_cast<float>(sqrt(total));
    if (rank == 0) *a.norm = s_norm;
  }
  if (!a.clip) return;
  __syncthreads();
  const float norm = s_norm;
  const float f = clip_factor(a.max_norm, norm, a.eps);
  int i = first < chunks ? locate(a, first) : 0;
  for (int c = first; c < chunks; c += kGroups) {
    while (c >= a.first[i + 1]) ++i;
    const Piece p = piece_of(a, i, c);
    uint4 w[kVecs];
    load_pieces(p, w);
    scale_chunk(p, w, f);
  }
}

// Starts while the launch before ends; the kernel waits for its results itself.
template <class... Params, class... Args>
cudaError_t launch_after(void (*kernel)(Params...), int grid, int threads, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool is_f32(const GradArgs& a, int i) { return a.dtypes[i] == kGradF32; }

int64_t chunks_of(const GradArgs& a, int i) {
  const int64_t bytes = a.sizes[i] * (is_f32(a, i) ? 4 : 2);
  int64_t skip = (16 - (reinterpret_cast<uintptr_t>(a.grads[i]) & 15)) & 15;
  if (skip > bytes) skip = bytes;
  const int64_t whole = (bytes - skip) & ~int64_t(15);
  if (bytes == 0) return 0;
  return whole > 0 ? (whole + kChunk - 1) / kChunk : 1;
}

// The tensors of one launch, their chunks, and its CTAs.
struct Group {
  int begin, end, grid;
  int64_t chunks;
};
Group group_from(const GradArgs& a, int begin) {
  Group g = {begin, begin, 0, 0};
  while (g.end < a.count && g.end - begin < kLargeTable) g.chunks += chunks_of(a, g.end++);
  const int64_t most = static_cast<int64_t>(a.sms < kMostSms ? a.sms : kMostSms) * kCtasPerSm;
  g.grid = static_cast<int>(g.chunks < 1 ? 1 : (g.chunks < most ? g.chunks : most));
  return g;
}

template <int CAP>
void fill(Table<CAP>* k, const GradArgs& a, const Group& g) {
  k->count = g.end - g.begin;
  int at = 0;
  for (uint32_t& w : k->f32) w = 0;
  for (int j = 0; j < k->count; ++j) {
    const int i = g.begin + j;
    k->t[j].g = a.grads[i];
    k->t[j].out = a.outs != nullptr ? a.outs[i] : const_cast<void*>(a.grads[i]);
    k->t[j].n = a.sizes[i];
    k->first[j] = at;
    at += static_cast<int>(chunks_of(a, i));
    if (is_f32(a, i)) k->f32[j >> 5] |= 1u << (j & 31);
  }
  k->first[k->count] = at;
  k->sums = a.sums;
  k->norm = g.begin == 0 ? a.norm : nullptr;
  k->norm_in = a.norm_in;
  k->max_norm = a.max_norm;
  k->eps = a.eps;
}

// One cluster, where the context can run it (asked once per context and thread).
template <int CAP>
bool launch_small(const Table<CAP>& k, cudaStream_t stream, cudaError_t* err) {
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int active = 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kSmallCluster);
  cfg.blockDim = dim3(kSmallThreads);
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = kSmallCluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if (asked_ctx == 0 || asked_ctx != current_context_id()) {
    if (cudaOccupancyMaxActiveClusters(&active, grad_small_kernel<CAP>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();  // a size that does not fit is no error of the call
      active = 0;
    }
    asked_ctx = current_context_id();
  }
  if (active < 1) return false;
  cfg.stream = stream;
  *err = cudaLaunchKernelEx(&cfg, grad_small_kernel<CAP>, k);
  return true;
}

// All tensors in one table.
template <int CAP>
cudaError_t launch_one(const GradArgs& a, const Group& g, bool clip, cudaStream_t stream) {
  Table<CAP> k;
  fill(&k, a, g);
  k.clip = clip;
  k.sums_at = 0;
  k.total = g.grid;
  cudaError_t err = cudaSuccess;
  if (a.norm_in == nullptr) {
    if (g.chunks <= kSmallChunks && a.max_cluster != 1 && launch_small<CAP>(k, stream, &err)) return err;
    err = launch_after(grad_norm_kernel<CAP>, g.grid, kThreads, stream, k);
    if (err != cudaSuccess) return err;
    if (!clip) return launch_after(grad_norm_end_kernel, 1, 32, stream, static_cast<const double*>(a.sums), g.grid, a.norm);
  }
  return launch_after(grad_clip_kernel<CAP>, g.grid, kThreads, stream, k);
}

// A table's worth of many tensors.
cudaError_t launch_part(const GradArgs& a, const Group& g, int sums_at, int total, bool clip, cudaStream_t stream) {
  Table<kLargeTable> k;
  fill(&k, a, g);
  k.sums_at = sums_at;
  k.total = total;
  if (clip) return launch_after(grad_clip_kernel<kLargeTable>, g.grid, kThreads, stream, k);
  return launch_after(grad_norm_kernel<kLargeTable>, g.grid, kThreads, stream, k);
}

}  // namespace

size_t grad_workspace_bytes(int count) {
  // a sum for every CTA of every launch
  const size_t launches = count > 0 ? (static_cast<size_t>(count) + kLargeTable - 1) / kLargeTable : 1;
  return sizeof(double) * launches * kMostSms * kCtasPerSm;
}

cudaError_t launch_grad(const GradArgs& a, bool clip, cudaStream_t stream) {
  if (a.count <= kLargeTable && (a.count > 0 || a.norm_in == nullptr)) {
    const Group g = group_from(a, 0);
    return a.count <= kSmallTable ? launch_one<kSmallTable>(a, g, clip && a.count > 0, stream)
                                  : launch_one<kLargeTable>(a, g, clip, stream);
  }
  int total = 0;
  if (a.norm_in == nullptr) {
    for (int i = 0; i < a.count;) {
      const Group g = group_from(a, i);
      const cudaError_t err = launch_part(a, g, total, 0, false, stream);
      if (err != cudaSuccess) return err;
      total += g.grid;
      i = g.end;
    }
    if (!clip) return launch_after(grad_norm_end_kernel, 1, 32, stream, static_cast<const double*>(a.sums), total, a.norm);
  }
  for (int i = 0; i < a.count;) {
    const Group g = group_from(a, i);
    const cudaError_t err = launch_part(a, g, 0, total, true, stream);
    if (err != cudaSuccess) return err;
    i = g.end;
  }
  return cudaSuccess;
}

}  // namespace mgw
