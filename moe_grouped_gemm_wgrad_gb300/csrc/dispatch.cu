// Row tables of routed tokens: a stable counting sort of the (token, slot) pairs by expert.
//
//   expert_off[e]  = pairs of experts below e
//   row_of[p]      = expert_off[e(p)] + pairs of e(p) before p   (-1 for a dropped pair)
//   row_index[r]   = p / top_k of the pair p with row_of[p] = r  (-1 past the last row)
//
// Every warp owns a contiguous run of pairs.  Pass 1 counts a run's experts in the warp's row
// of shared memory; a scan over runs and experts turns the counts into every run's first row
// per expert; pass 2 walks the run again, 32 pairs at a time, a pair's rank among equal
// experts of the 32 coming from one warp match.  No atomics decide an order: the rows of an
// expert are its pairs in ascending order, on every run.
//
// Up to kSmallPairs pairs one CTA does it all in one launch (12 bytes a pair: latency bounds
// it).  More pairs go to `blocks` CTAs in two launches: CTA counts to the workspace, then each
// CTA sums the counts of the CTAs before it and places its own pairs.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kSmallPairs = 8192;
constexpr int kPairsPerBlock = 8192;
constexpr int kMaxBlocks = 128;

// Warps per CTA: their E counters each share 64 KB.
constexpr int warps_for(int E) { return E <= 512 ? 32 : 16; }

// The pair's expert, or -1 for a dropped one; anything else outside the range is reported.
__device__ __forceinline__ int expert_of(const DispatchArgs& a, int p) {
  int e = a.expert_idx[p];
  if (e < -1 || e >= a.E) {
    if (a.status != nullptr) atomicOr(a.status, kDevBadIndex);
    e = -1;
  }
  return e;
}

// This CTA's pairs [lo, hi) and its warp's part of them (whole groups of 32 per warp).
struct Run {
  int lo, hi;
};
__device__ __forceinline__ Run block_run(const DispatchArgs& a, int b, int blocks) {
  const int per = (a.pairs / 32 + blocks) / blocks * 32;
  Run r;
  const long long lo = static_cast<long long>(b) * per;
  r.lo = static_cast<int>(lo < a.pairs ? lo : a.pairs);
  r.hi = static_cast<int>(lo + per < a.pairs ? lo + per : a.pairs);
  return r;
}
__device__ __forceinline__ Run warp_run(Run b, int w, int warps) {
  const int per = ((b.hi - b.lo + 31) / 32 + warps - 1) / warps * 32;
  Run r;
  const long long lo = b.lo + static_cast<long long>(w) * per;
  r.lo = static_cast<int>(lo < b.hi ? lo : b.hi);
  r.hi = static_cast<int>(lo + per < b.hi ? lo + per : b.hi);
  return r;
}

// Counts the run's experts into cnt[0 .. E), which is zero.
__device__ __forceinline__ void count_run(const DispatchArgs& a, Run r, int* cnt) {
  const int lane = static_cast<int>(lane_id());
  for (int p0 = r.lo; p0 < r.hi; p0 += 32) {
    const int p = p0 + lane;
    const int e = p < r.hi ? expert_of(a, p) : -1;
    if (e >= 0) atomicAdd(&cnt[e], 1);
  }
}

// Places the run's pairs; next[e] is the run's next row of expert e.
__device__ __forceinline__ void place_run(const DispatchArgs& a, Run r, int* next) {
  const int lane = static_cast<int>(lane_id());
  for (int p0 = r.lo; p0 < r.hi; p0 += 32) {
    const int p = p0 + lane;
    const bool in = p < r.hi;
    int e = in ? a.expert_idx[p] : -1;
    if (e >= a.E) e = -1;
    const unsigned same = __match_any_sync(kAll, e);
    int row = -1;
    if (e >= 0) row = next[e] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (e >= 0 && lane == 31 - __clz(same)) next[e] = row + 1;
    __syncwarp();
    if (in) a.row_of[p] = row;
    if (row >= 0) a.row_index[row] = p / a.top_k;
  }
}

// Turns per-warp counts [warps][E] into first rows: row of (w, e) = base[e] + counts of e in
// the warps below w.  Returns e's total over the warps.
__device__ __forceinline__ int scan_warps(int* cnt, int warps, int E, int e, int base) {
  int run = base;
  for (int w = 0; w < warps; ++w) {
    const int c = cnt[w * E + e];
    cnt[w * E + e] = run;
    run += c;
  }
  return run - base;
}

// Exclusive scan of s[0 .. E) in place by one warp, s[E] = the total.
__device__ __forceinline__ void warp_scan(int* s, int E) {
  const int lane = static_cast<int>(lane_id());
  int carry = 0;
  for (int base = 0; base < E; base += 32) {
    const int e = base + lane;
    const int c = e < E ? s[e] : 0;
    int v = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(kAll, v, d);
      if (lane >= d) v += y;
    }
    if (e < E) s[e] = carry + v - c;
    carry += __shfl_sync(kAll, v, 31);
  }
  if (lane == 0) s[E] = carry;
}

__global__ void __launch_bounds__(1024) dispatch_small_kernel(DispatchArgs a) {
  extern __shared__ int s_cnt[];  // [warps][E], then the E + 1 offsets
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  int* s_off = s_cnt + warps * a.E;
  for (int i = threadIdx.x; i < warps * a.E; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  const Run b{0, a.pairs};
  const Run r = warp_run(b, warp, warps);
  count_run(a, r, s_cnt + warp * a.E);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) s_off[e] = scan_warps(s_cnt, warps, a.E, e, 0);
  __syncthreads();
  if (warp == 0) warp_scan(s_off, a.E);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.expert_off[e] = s_off[e];
  for (int i = threadIdx.x; i < warps * a.E; i += blockDim.x) s_cnt[i] += s_off[i % a.E];
  for (int i = s_off[a.E] + threadIdx.x; i < a.pairs; i += blockDim.x) a.row_index[i] = -1;
  __syncthreads();
  place_run(a, r, s_cnt + warp * a.E);
}

__global__ void __launch_bounds__(1024) dispatch_count_kernel(DispatchArgs a) {
  extern __shared__ int s_cnt[];  // [E]
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  count_run(a, warp_run(block_run(a, blockIdx.x, gridDim.x), warp, warps), s_cnt);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    a.counts[static_cast<size_t>(blockIdx.x) * a.E + e] = s_cnt[e];
}

__global__ void __launch_bounds__(1024) dispatch_place_kernel(DispatchArgs a) {
  extern __shared__ int s_cnt[];  // [warps][E], the E + 1 offsets, this CTA's first rows [E]
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
  int* s_off = s_cnt + warps * a.E;
  int* s_base = s_off + a.E + 1;
  for (int i = threadIdx.x; i < warps * a.E; i += blockDim.x) s_cnt[i] = 0;
  // totals over all CTAs, and over the CTAs before this one
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
    int before = 0, all = 0;
    for (unsigned b = 0; b < gridDim.x; ++b) {
      const int c = a.counts[static_cast<size_t>(b) * a.E + e];
      all += c;
      if (b < blockIdx.x) before += c;
    }
    s_off[e] = all;
    s_base[e] = before;
  }
  __syncthreads();
  const Run r = warp_run(block_run(a, blockIdx.x, gridDim.x), warp, warps);
  count_run(a, r, s_cnt + warp * a.E);
  if (warp == 0) {
    __syncwarp();
    warp_scan(s_off, a.E);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    (void)scan_warps(s_cnt, warps, a.E, e, s_off[e] + s_base[e]);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.expert_off[e] = s_off[e];
  for (long long i = s_off[a.E] + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.pairs;
       i += static_cast<long long>(gridDim.x) * blockDim.x)
    a.row_index[i] = -1;
  __syncthreads();
  place_run(a, r, s_cnt + warp * a.E);
}

size_t place_smem_bytes(int E) {
  return sizeof(int) * (static_cast<size_t>(warps_for(E)) * E + 2 * static_cast<size_t>(E) + 1);
}

}  // namespace

int dispatch_blocks(long long pairs, int E) {
  (void)E;
  if (pairs <= kSmallPairs) return 1;
  const long long b = (pairs + kPairsPerBlock - 1) / kPairsPerBlock;
  return static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
}

cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t stream) {
  const int blocks = dispatch_blocks(a.pairs, a.E);
  const int threads = 32 * warps_for(a.E);
  const size_t smem = place_smem_bytes(a.E);
  static thread_local uint64_t attr_small = 0, attr_place = 0;
  const size_t max_smem = place_smem_bytes(512) > place_smem_bytes(kMaxExperts) ? place_smem_bytes(512)
                                                                                : place_smem_bytes(kMaxExperts);
  if (blocks == 1) {
    const cudaError_t err = set_smem_attr_once(reinterpret_cast<const void*>(dispatch_small_kernel),
                                               max_smem, &attr_small);
    if (err != cudaSuccess) return err;
    dispatch_small_kernel<<<1, threads, smem, stream>>>(a);
    return cudaGetLastError();
  }
  const cudaError_t err = set_smem_attr_once(reinterpret_cast<const void*>(dispatch_place_kernel),
                                             max_smem, &attr_place);
  if (err != cudaSuccess) return err;
  dispatch_count_kernel<<<blocks, threads, sizeof(int) * a.E, stream>>>(a);
  const cudaError_t e1 = cudaGetLastError();
  if (e1 != cudaSuccess) return e1;
  dispatch_place_kernel<<<blocks, threads, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace mgw
