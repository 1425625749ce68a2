// Row tables of routed tokens: a stable counting sort of the (token, slot) pairs by expert.
//
//   expert_off[e]  = pairs of experts below e
//   row_of[p]      = expert_off[e(p)] + pairs of e(p) before p   (-1 for a dropped pair)
//   row_index[r]   = p / top_k of the pair p with row_of[p] = r  (-1 past the last row)
//
// Every warp owns a contiguous run of pairs and a row of E counters in shared memory.  32 pairs
// at a time, ballots find the lanes of equal experts, and the last of them adds their
// number to the counter: the old value plus the lanes before is a pair's rank in the run.  A scan
// over the runs and over the experts then gives every run's first row per expert.  No atomic
// decides an order: the rows of an expert are its pairs in ascending order, on every run.
//
// Up to two groups of 32 pairs per warp one CTA does it all.  Up to 65536 pairs (32768 of more
// than 512 experts) a cluster of up to 16 CTAs does, whose CTAs read each other's counts from
// shared memory: one launch and no workspace.  More pairs go to more CTAs in two launches: CTA
// counts to the workspace, then each CTA ranks its own pairs, adds up the counts of the CTAs
// before it and stores.  12 bytes a pair are far from bounding it (1M pairs: 2 us); what does is
// the chain of phases within a CTA, so a CTA gets few pairs (up to eight groups a warp, whose
// experts and ranks then stay in registers).  128 pairs take 5 us, 65536 11, 1M pairs 19 (of 512
// experts 28).  The cluster takes as long as the two launches did, but the call returns 4.5 us
// sooner: 18 instead of 22.5 us a call at 65536.  Where a context cannot run 16 CTAs as a cluster
// (a share of the SMs), eight take the same calls with up to eight groups a warp, or one CTA does
// in two passes: 65536 pairs of 64 experts 9, 13 and 82 us, 16384 pairs 6, 7 and 23.
#include <cuda_runtime.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kHeld = 8;        // groups of 32 pairs a warp keeps in registers
constexpr int kMaxBlocks = 1024;
constexpr int kCluster = 16;    // CTAs of the one-launch form, at most
constexpr int kClusterGroups = 4;  // groups of 32 pairs a warp takes in it, at most
enum Mode { kOne, kClustered, kMany };

// Warps per CTA: their E counters each share 64 KB.
__host__ __device__ constexpr int warps_for(int E) { return E <= 512 ? 32 : 16; }
// Counters of a warp lie this far apart (odd: a column of them falls into different banks).
__host__ __device__ constexpr int stride_for(int E) { return E | 1; }

// The pair's expert, or -1 for a dropped one; anything else outside the range is reported.
__device__ __forceinline__ int expert_of(const DispatchArgs& a, int p) {
  int e = a.expert_idx[p];
  if (e < -1 || e >= a.E) {
    if (a.status != nullptr) atomicOr(a.status, kDevBadIndex);
    e = -1;
  }
  return e;
}

struct Run {
  int lo, hi;
};
// The i-th of n runs of whole groups of 32 pairs within [lo, hi).
__device__ __forceinline__ Run part(Run all, int i, int n) {
  const int per = ((all.hi - all.lo + 31) / 32 + n - 1) / n * 32;
  const long long lo = all.lo + static_cast<long long>(i) * per;
  Run r;
  r.lo = static_cast<int>(lo < all.hi ? lo : all.hi);
  r.hi = static_cast<int>(lo + per < all.hi ? lo + per : all.hi);
  return r;
}

// The lanes whose expert equals this lane's (of those with one): a ballot per bit of an expert's
// number.  The hardware's warp match goes through the distinct values one by one instead: with
// it a CTA's ranking takes longer the more experts there are (1M pairs of 512: 4 us longer).
__device__ __forceinline__ unsigned equal_lanes(int e, int bits) {
  unsigned same = __ballot_sync(kAll, e >= 0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (e >> b) & 1;
    const unsigned with = __ballot_sync(kAll, one);
    same &= one ? with : ~with;
  }
  return e >= 0 ? same : 1u << lane_id();
}

// Adds the group's experts to the counters; returns the lane's rank among the run's pairs of its
// expert (old counter value plus equal lanes before it).
__device__ __forceinline__ int rank_group(int e, int bits, int* cnt) {
  const int lane = static_cast<int>(lane_id());
  const unsigned same = equal_lanes(e, bits);
  const int last = 31 - __clz(same);
  int old = 0;
  if (e >= 0 && lane == last) {
    old = cnt[e];
    cnt[e] = old + __popc(same);
  }
  __syncwarp();
  old = __shfl_sync(kAll, old, last);
  return old + __popc(same & ((1u << lane) - 1u));
}

// Turns column e of the counters [warps][stride] into exclusive sums over the warps, one warp
// per column, lane w the w-th counter; the total comes back in every lane.
__device__ __forceinline__ int scan_column(int* cnt, int warps, int stride, int e) {
  const int lane = static_cast<int>(lane_id());
  const int c = lane < warps ? cnt[lane * stride + e] : 0;
  int v = c;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(kAll, v, d);
    if (lane >= d) v += y;
  }
  if (lane < warps) cnt[lane * stride + e] = v - c;
  return __shfl_sync(kAll, v, 31);
}

// Exclusive scan of s[0 .. E) in place by the block, s[E] = the total; s_seg holds 32 ints.
// Ends with a barrier.
__device__ __forceinline__ void block_scan(int* s, int E, int* s_seg) {
  const int lane = static_cast<int>(lane_id()), warps = blockDim.x >> 5;
  const int segs = (E + 31) / 32;  // of 32 experts, at most 32
  for (int g = threadIdx.x >> 5; g < segs; g += warps) {
    const int e = 32 * g + lane;
    const int c = e < E ? s[e] : 0;
    int v = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(kAll, v, d);
      if (lane >= d) v += y;
    }
    if (e < E) s[e] = v - c;
    if (lane == 31) s_seg[g] = v;
  }
  __syncthreads();
  for (int g = threadIdx.x >> 5; g < segs; g += warps) {
    const int before = __reduce_add_sync(kAll, lane < g ? s_seg[lane] : 0);
    const int e = 32 * g + lane;
    if (e < E) s[e] += before;
    if (g == segs - 1 && lane == 0) s[E] = before + s_seg[g];
  }
  __syncthreads();
}

// This CTA's pair counts per expert.
__global__ void __launch_bounds__(1024) dispatch_count_kernel(DispatchArgs a) {
  extern __shared__ int s_cnt[];  // [E]
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int warps = blockDim.x >> 5, lane = static_cast<int>(lane_id());
  const int bits = 32 - __clz(a.E - 1);
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) s_cnt[i] = 0;
  __syncthreads();
  const Run r = part(part(Run{0, a.pairs}, blockIdx.x, gridDim.x), threadIdx.x >> 5, warps);
  for (int p0 = r.lo; p0 < r.hi; p0 += 32 * kHeld) {
    int e[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int p = p0 + 32 * i + lane;
      e[i] = p < r.hi ? expert_of(a, p) : -1;
    }
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const unsigned same = equal_lanes(e[i], bits);
      if (e[i] >= 0 && lane == 31 - __clz(same)) atomicAdd(&s_cnt[e[i]], __popc(same));
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += blockDim.x)
    a.counts[static_cast<size_t>(blockIdx.x) * a.E + e] = s_cnt[e];
}

__device__ __forceinline__ int ld_cluster(uint32_t cluster_addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}

// Ranks and places this CTA's pairs.  kOne: the only CTA, whose counts are the totals.
// kClustered: the grid is one cluster, whose CTAs read each other's counts from shared memory.
// kMany: all CTAs' counts are in the workspace.  HELD: a warp's run is at most kHeld groups.
template <Mode MODE, bool HELD>
__global__ void __launch_bounds__(1024) dispatch_place_kernel(DispatchArgs a) {
  // counters [warps][stride], expert offsets [E + 1], first rows [E], this CTA's counts [E]
  extern __shared__ int s_cnt[];
  __shared__ int s_seg[32];
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = static_cast<int>(lane_id());
  const int stride = stride_for(a.E), bits = 32 - __clz(a.E - 1);
  int* s_off = s_cnt + warps * stride;
  int* s_first = s_off + a.E + 1;
  int* s_mine = s_first + a.E;
  int* mine = s_cnt + warp * stride;
  for (int i = threadIdx.x; i < warps * stride; i += blockDim.x) s_cnt[i] = 0;
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) s_off[e] = s_first[e] = 0;
  const Run r = part(part(Run{0, a.pairs}, blockIdx.x, gridDim.x), warp, warps);
  int ex[kHeld], rank[kHeld];
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int p = r.lo + 32 * i + lane;
      ex[i] = p < r.hi ? expert_of(a, p) : -1;
    }
  }
  __syncthreads();
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (r.lo + 32 * i < r.hi) rank[i] = rank_group(ex[i], bits, mine);
  } else {
    for (int p0 = r.lo; p0 < r.hi; p0 += 32)
      (void)rank_group(p0 + lane < r.hi ? expert_of(a, p0 + lane) : -1, bits, mine);
  }
  __syncthreads();
  for (int e = warp; e < a.E; e += warps) {
    const int total = scan_column(s_cnt, warps, stride, e);
    if (MODE == kOne && lane == 0) s_off[e] = total;
    if (MODE == kClustered && lane == 0) s_mine[e] = total;
  }
  if constexpr (MODE == kClustered) {
    cluster_sync();  // every CTA's counts are there
    const int blocks = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) {
      int c[kCluster], all = 0, before = 0;
#pragma unroll
      for (int b = 0; b < kCluster; ++b)
        c[b] = b < blocks ? ld_cluster(map_to_cta(smem_u32(s_mine + e), static_cast<uint32_t>(b))) : 0;
#pragma unroll
      for (int b = 0; b < kCluster; ++b) {
        all += c[b];
        before += b < me ? c[b] : 0;
      }
      s_off[e] = all;
      s_first[e] = before;
    }
    // read; waited for before the CTA ends
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  }
  if constexpr (MODE == kMany) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the counting launch has finished
    // Totals over all CTAs, and over the CTAs before this one: every thread adds up a share of
    // one expert's column (integer sums, whose order does not matter).
    const int blocks = static_cast<int>(gridDim.x), me = static_cast<int>(blockIdx.x);
    const int parts = max(static_cast<int>(blockDim.x) / a.E, 1);
    for (int i = threadIdx.x; i < parts * a.E; i += blockDim.x) {
      const int e = i % a.E;
      int all = 0, before = 0;
#pragma unroll 8
      for (int b = i / a.E; b < blocks; b += parts) {
        const int c = a.counts[static_cast<size_t>(b) * a.E + e];
        all += c;
        before += b < me ? c : 0;
      }
      atomicAdd(&s_off[e], all);
      atomicAdd(&s_first[e], before);
    }
  }
  __syncthreads();
  block_scan(s_off, a.E, s_seg);
  for (int e = threadIdx.x; e < a.E; e += blockDim.x) s_first[e] += s_off[e];
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += blockDim.x) a.expert_off[e] = s_off[e];
  for (long long i = s_off[a.E] + static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < a.pairs;
       i += static_cast<long long>(gridDim.x) * blockDim.x)
    a.row_index[i] = -1;
  __syncthreads();
  // the token p / top_k of this lane's pair, carried along from group to group of 32
  int token = (r.lo + lane) / a.top_k, slot = (r.lo + lane) % a.top_k;
  const int tokens32 = 32 / a.top_k, slots32 = 32 % a.top_k;
  auto place = [&](int p, int e, int row) {
    if (p < r.hi) a.row_of[p] = e >= 0 ? row : -1;
    if (e >= 0) a.row_index[row] = token;
    token += tokens32;
    slot += slots32;
    if (slot >= a.top_k) slot -= a.top_k, ++token;
  };
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      if (r.lo + 32 * i < r.hi) {
        const int e = ex[i];
        place(r.lo + 32 * i + lane, e, e >= 0 ? s_first[e] + mine[e] + rank[i] : -1);
      }
    }
  } else {
    // the counters now hold the run's first rows: ranking again gives the rows
    for (int p0 = r.lo; p0 < r.hi; p0 += 32) {
      int e = p0 + lane < r.hi ? a.expert_idx[p0 + lane] : -1;
      if (e >= a.E || e < 0) e = -1;
      const int rank = rank_group(e, bits, mine);
      place(p0 + lane, e, e >= 0 ? s_first[e] + rank : -1);
    }
  }
  if constexpr (MODE == kClustered) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

size_t place_smem_bytes(int E) {
  return sizeof(int) * (static_cast<size_t>(warps_for(E)) * stride_for(E) + 3 * static_cast<size_t>(E) + 1);
}

size_t max_place_smem() {
  return place_smem_bytes(512) > place_smem_bytes(kMaxExperts) ? place_smem_bytes(512)
                                                               : place_smem_bytes(kMaxExperts);
}

// The largest cluster, of 16 or 8 CTAs, that the current context can run; 1 when it can run
// neither (a process may have a share of the SMs only).  Asked once per context and thread.
int largest_cluster() {
  static thread_local uint64_t attr_ctx = 0;
  static thread_local int largest = 0;
  if (attr_ctx != 0 && attr_ctx == current_context_id()) return largest;
  const void* kernel = reinterpret_cast<const void*>(dispatch_place_kernel<kClustered, true>);
  largest = 1;
  // clusters of more than eight CTAs have to be asked for, once per context as well
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      set_smem_attr_once(kernel, max_place_smem(), &attr_ctx) == cudaSuccess) {
    for (int size = kCluster; size >= 8 && largest == 1; size /= 2) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(size));
      cfg.blockDim = dim3(1024);
      cfg.dynamicSmemBytes = max_place_smem();
      cudaLaunchAttribute attr = {};
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = static_cast<unsigned>(size);
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int active = 0;
      if (cudaOccupancyMaxActiveClusters(&active, kernel, &cfg) != cudaSuccess)
        (void)cudaGetLastError();  // a size that does not fit is no error of the call
      else if (active > 0)
        largest = size;
    }
  }
  return largest;
}

template <Mode MODE, bool HELD>
cudaError_t launch_place(const DispatchArgs& a, int blocks, cudaStream_t stream) {
  static thread_local uint64_t attr_ctx = 0;
  const void* kernel = reinterpret_cast<const void*>(dispatch_place_kernel<MODE, HELD>);
  const cudaError_t err = set_smem_attr_once(kernel, max_place_smem(), &attr_ctx);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps_for(a.E)));
  cfg.dynamicSmemBytes = place_smem_bytes(a.E);
  cfg.stream = stream;
  cudaLaunchAttribute attr = {};
  if (MODE == kClustered) {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(blocks);
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
  } else {
    // After a counting launch, the placing one starts while that runs (programmatic dependent
    // launch): it ranks its own pairs, and waits before it reads the table or writes anything.
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = MODE == kOne ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, dispatch_place_kernel<MODE, HELD>, a);
}

// CTAs of a cluster of at most `most` CTAs that take up to `groups` groups a warp (one, two, four ..);
// 0 for more pairs than that.
int cluster_blocks(long long pairs, int E, int most, int groups) {
  const long long group = 32 * warps_for(E);  // pairs of one group per warp
  for (int g = 1; g <= groups; g *= 2)
    if (pairs <= most * g * group) return static_cast<int>((pairs + g * group - 1) / (g * group));
  return 0;
}

// CTAs of a call that one launch does: one, or a cluster; 0 for calls that take two launches.
int one_launch_blocks(long long pairs, int E) {
  if (pairs <= 2 * 32 * warps_for(E)) return 1;
  return cluster_blocks(pairs, E, kCluster, kClusterGroups);
}

// CTAs of the two launches.
int many_blocks(long long pairs, int E) {
  const long long group = 32 * warps_for(E);
  // one, two, four or eight groups a warp while that keeps the CTAs to the device's size
  for (int g = 1; g < kHeld; g *= 2)
    if (pairs <= 128 * g * group) return static_cast<int>((pairs + g * group - 1) / (g * group));
  const long long b = (pairs + kHeld * group - 1) / (kHeld * group);
  return static_cast<int>(b < kMaxBlocks ? b : kMaxBlocks);
}

}  // namespace

size_t dispatch_workspace_bytes(long long pairs, int E) {
  if (one_launch_blocks(pairs, E) > 0) return 0;
  return sizeof(int) * static_cast<size_t>(many_blocks(pairs, E)) * static_cast<size_t>(E);
}

cudaError_t launch_dispatch(const DispatchArgs& a, cudaStream_t stream) {
  const int few = one_launch_blocks(a.pairs, a.E);
  if (few == 1) return launch_place<kOne, true>(a, 1, stream);
  if (few > 1) {
    int most = largest_cluster();
    if (a.max_cluster > 0 && a.max_cluster < most) most = a.max_cluster;
    if (few <= most) return launch_place<kClustered, true>(a, few, stream);
    // Clusters of eight take the same calls with twice the groups a warp.  Without clusters one
    // CTA takes them all: these calls have no workspace for the two launches.
    const int blocks = cluster_blocks(a.pairs, a.E, most, kHeld);
    return blocks > 1 ? launch_place<kClustered, true>(a, blocks, stream) : launch_place<kOne, false>(a, 1, stream);
  }
  const int blocks = many_blocks(a.pairs, a.E);
  const int threads = 32 * warps_for(a.E);
  dispatch_count_kernel<<<blocks, threads, sizeof(int) * a.E, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  const long long groups = (static_cast<long long>(a.pairs) + 31) / 32;
  const bool held = (groups + blocks - 1) / blocks <= static_cast<long long>(kHeld) * warps_for(a.E);
  return held ? launch_place<kMany, true>(a, blocks, stream) : launch_place<kMany, false>(a, blocks, stream);
}

}  // namespace mgw
