// Gradients of the low-rank adapters: for the rows r of adapter e
//
//   dA[e][j][k] = scale[e] sum_r v[r][j] x[t(r)][k]      dB[e][n][j] = scale[e] sum_r dy[o(r)][n] u[r][j]
//
// Both are grad = X^T Q, X bf16 rows contracted over the rows (as an expert's weight gradient is), Q
// rank-wide.  X's rows arrive as they lie in memory, 64 tokens by 64 features, and the tensor core
// reads them across (MN-major, see lora.cuh): nothing is transposed.  Q comes from the data gradient's
// launch in blocks of 64 tokens, already scaled, split into two bf16 parts (split2) and laid out as
// the operand tile that the tensor core reads: one bulk copy each.  Both parts go through one product of
// twice the rank's width and are added up in the epilogue.
//
// A cluster has 256 features of one of the two gradients and all token blocks, of all adapters one
// after the other, in equal shares: however unevenly the rows fall on the adapters, the CTAs have
// the same work.  An adapter whose blocks lie in one share is stored from TMEM; one that shares divide
// is written as fp32 partial sums to the workspace, and behind a cluster barrier its CTAs add them up
// in the order of the shares, a part of the features each.  No atomics, no second launch, the same
// bits on every run.
//
// HBM bounds it: dy and x once.  16384 rows of one adapter, 4096 and 4096 features, rank 64: 53 us,
// 5.1 TB/s; 8192 rows of 16 adapters, scattered, 8192 and 4096 features, rank 16: 49 us, 4.1 TB/s (96 CTAs:
// 48 feature blocks fit two to a cluster).  Shares of all 152 SMs that cross the feature blocks' borders,
// their sums added up by the last CTA to come, took 6 us off the latter, but 4 to 19 us more with 64
// feature blocks (8192 rows, ranks 16 to 128) and half as much again with 1024 rows of 14 (rank 128).
//
// Roles (448 threads): warp 0 loads by TMA, warps 6-13 copy rows that lie apart and an adapter's last rows
// (four warps, too few loads in flight, took 4 us more for 8192 scattered rows) and then zero the gradients
// of adapters without rows, warp 1 issues the MMAs, warps 2-5 are the epilogue, which overlaps the next
// adapter's blocks where two accumulators fit into TMEM (rank up to 64).
#include <cuda_runtime.h>

#include <cstdint>

#include "lora.cuh"

namespace mgw {
namespace {

using namespace lora;

constexpr int kThreads = 448;
constexpr int kTok = 64;           // tokens per stage
constexpr int kWidth = 256;        // features per CTA
constexpr int kXBytes = 4 * 8192;  // 64 tokens of 256 features
constexpr int kMaxStages = 6;
constexpr int kMaxCluster = 8;
// Token blocks that one accumulator takes.  The tensor core cuts each addition's low bits off, always
// downwards: of a sum that only grows 1.1e-7 an addition, one for every 16 rows.  In one accumulator a
// million rows came out 0.7% too small, four million 2.8%; 16384 rows are off by 1e-4, where half a step of a
// bf16 gradient is 2e-3 to 4e-3.  Longer runs are added up in fp32 in the workspace: the sums of 256 features
// (64 KB at rank 64) read and written once for every 8 MB of X.  65536 rows, 8192 and 8192 features, rank 64:
// backward 832 -> 836 us, rank 128 1028 -> 1038 (there is one accumulator, and the products wait for it).
constexpr int kChain = 256;
constexpr int kSms = 152;          // of a GB300: the workspace's size has no device to ask
constexpr int kBarBytes = 8 * (2 * kMaxStages + 4);

__host__ __device__ constexpr int padded_rank(int R) { return (R + 15) & ~15; }
__host__ __device__ constexpr int stage_bytes(int RP) { return kXBytes + 256 * RP; }
constexpr size_t misc_bytes(int E) { return kBarBytes + 16 + sizeof(int) * (static_cast<size_t>(E) + 1) + 1024; }
constexpr int stages_of(int RP) {
  const int n = static_cast<int>((227 * 1024 - misc_bytes(kMaxExperts)) / stage_bytes(RP));
  return n < kMaxStages ? n : kMaxStages;
}
static_assert(stages_of(128) == 3 && stages_of(64) == 4 && stages_of(16) == 6, "ring");
constexpr size_t part_floats(int RP) { return static_cast<size_t>(kWidth) * RP; }

// The share of the token blocks of CTA p of C.  (At most 2^25 + 1024 blocks, C at most 8.)
__device__ __forceinline__ int share(int blocks, int p, int C) {
  return static_cast<int>(static_cast<uint32_t>(blocks) * static_cast<uint32_t>(p) / static_cast<uint32_t>(C));
}

__global__ void __launch_bounds__(kThreads, 1) lora_grad_kernel(const __grid_constant__ LoraGradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t lane = lane_id();
  const int C = a.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int E = a.E, R = a.R, RP = padded_rank(R);
  const int S = a.stages;
  uint8_t* bars = smem + S * stage_bytes(RP);
  int* s_misc = reinterpret_cast<int*>(bars + kBarBytes);  // [0] TMEM [1] abort [2] token blocks
  int* s_off = s_misc + 4;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(s_misc + 1);
  int item = static_cast<int>(blockIdx.x) / C;
  const int which = item >= a.first1 ? 1 : 0;
  if (which) item -= a.first1;
  const LoraGradJob& job = a.job[which];
  const int cols = job.cols, f0 = item * kWidth;

  const uint32_t bar0 = smem_u32(bars);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto bar_acc = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
  auto bar_free = [&](int s) { return bar0 + 8u * (2 * kMaxStages + 2 + s); };
  if (tid == 0) {
    tma_prefetch_desc(&job.tm);
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_full(s), 1 + 256);
      mbar_init(bar_empty(s), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_acc(s), 1);
      mbar_init(bar_free(s), 4);
    }
    fence_mbar_init();
    s_misc[1] = 0;
    s_misc[2] = 0;
  }
  for (int i = tid; i <= E; i += kThreads) s_off[i] = a.off[i];
  __syncthreads();
  int bad = 0, mine = 0;
  for (int i = tid; i < E; i += kThreads) {
    // compared, not subtracted: the difference of offsets that are none may wrap to a positive number
    bad |= s_off[i + 1] < s_off[i];
    mine += (s_off[i + 1] - s_off[i] + kTok - 1) / kTok;
  }
  if (tid == 0) bad |= s_off[0] != 0 || s_off[E] > a.M;
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) atomicAdd(&s_misc[2], mine);
  if (__syncthreads_or(bad)) {
    if (tid == 0 && a.status != nullptr) atomicOr(a.status, kDevBadOffsets);
    wait_for_launch_before();
    return;
  }
  const int blocks = s_misc[2];
  const int t0 = share(blocks, rank, C), t1 = share(blocks, rank + 1, C);
  const uint32_t tmem_cols = RP <= 16 ? 128u : (RP <= 32 ? 256u : 512u);
  const int bufs = RP <= 64 ? 2 : 1;
  if (warp == 1) {
    tmem_alloc(smem_u32(s_misc), tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_misc[0]);

  // Walks the adapters' token blocks in this CTA's share, one adapter at a time.
  struct Walk {
    const int* off;
    int e, at, pad;  // adapter, its first block (counted over all), its first row tile of 128
    int lo, n;       // its rows
    int b0, b1;      // its blocks within the share, counted within the adapter
    __device__ __forceinline__ bool next(int t0, int t1, int E) {
      if (t0 >= t1) return false;
      while (++e < E) {
        at += (n + kTok - 1) / kTok;
        pad += (n + 127) / 128;
        lo = off[e];
        n = off[e + 1] - lo;
        const int end = at + (n + kTok - 1) / kTok;
        if (at >= t1) return false;
        if (n > 0 && end > t0) {
          b0 = max(t0 - at, 0);
          b1 = min(t1, end) - at;
          return true;
        }
      }
      return false;
    }
  };
  Walk w = {s_off, -1, 0, 0, 0, 0, 0, 0};
  // Rows behind an adapter's last one must be zeros (their products with Q's zeros would not be 0
  // for infinities): only whole blocks come as one box.
  auto in_box = [&](int left) { return job.index == nullptr && left >= kTok; };

  __nv_bfloat16* grad = static_cast<__nv_bfloat16*>(job.grad);
  if (warp == 0) {
    // ------------------------------------------------------------ producer
    bool ok = true;
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    while (ok && w.next(t0, t1, E)) {
      for (int b = w.b0; b < w.b1; ++b) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_empty(stage), phase ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          const bool box = in_box(w.n - b * kTok);
          const uint32_t fb = bar_full(stage), sx = sbase + stage * stage_bytes(RP), q_bytes = 256u * RP;
          mbar_arrive_expect_tx(fb, (box ? static_cast<uint32_t>(kXBytes) : 0u) + q_bytes);
          if (box) {
#pragma unroll
            for (int k = 0; k < 4; ++k) tma_load_2d(sx + k * 8192, &job.tm, f0 + 64 * k, w.lo + b * kTok, fb);
          }
          // Q comes from the launch before, X does not
          if (filled == 0) wait_for_launch_before();
          bulk_load(sx + kXBytes, job.q + (2ll * w.pad + b) * q_bytes, q_bytes, fb);
        }
        __syncwarp();
        ++filled;
        if (++stage == S) stage = 0, phase ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    // Never leave the CTA with copies still landing in shared memory.
    for (int i = filled > S ? filled - S : 0; i < filled; ++i) mbar_wait_drain(bar_full(i % S), (i / S) & 1u);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const bool issue = elect_one();
    const uint32_t idesc = idesc_bf16(2 * RP, true, false);
    bool ok = true;
    int stage = 0, i = 0;
    uint32_t phase = 0;
    while (ok && w.next(t0, t1, E)) {
      for (int c0 = w.b0; ok && c0 < w.b1; c0 += kChain, ++i) {
        const int c1 = min(w.b1, c0 + kChain);
        const int buf = bufs == 2 ? i & 1 : 0, use = bufs == 2 ? i >> 1 : i;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_free(buf), (use & 1) ^ 1u, abort_flag));
        const uint32_t d = tmem + static_cast<uint32_t>(buf * 4 * RP);
        for (int b = c0; ok && b < c1; ++b) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar_full(stage), phase, abort_flag));
          if (!ok) break;
          fence_async_smem();  // copied rows are generic writes
          tc_fence_after();
          const uint32_t sx = sbase + stage * stage_bytes(RP);
          const int steps = (min(kTok, w.n - b * kTok) + 15) >> 4;
          if (issue) {
            const uint64_t bd = sdesc_kmajor_sw128(sx + kXBytes);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint64_t ad = sdesc_mn_sw128(sx + h * 16384, 8192);
              for (int k = 0; k < steps; ++k)
                mma_bf16(d + h * 2 * RP, ad + kStepMn * k, bd + kStepK * k, idesc, b != c0 || k != 0);
            }
            mma_commit(bar_empty(stage));
          }
          __syncwarp();
          if (++stage == S) stage = 0, phase ^= 1u;
        }
        if (ok && issue) mma_commit(bar_acc(buf));
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    // All MMAs have completed before TMEM is released: the epilogue waits for every accumulator but
    // one that a time-out cut short.
    if (!ok && issue) {
      mma_commit(bar_acc(0));
      mma_commit(bar_acc(1));
    }
    __syncwarp();
  } else if (warp >= 6) {
    // ------------------------------------------------- rows that lie apart
    // A warp has 8 of a block's tokens, all lanes one row at a time (512 bytes).  Blocks that come
    // as a box it only passes on, in step.
    const int q0 = (warp - 6) * 8, ch = static_cast<int>(lane & 7);
    const uint32_t part = (lane >> 3) * 8192u;
    const int col = f0 + 8 * static_cast<int>(lane);
    const bool there = col < cols;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(job.x) + (there ? col : 0);
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    while (ok && w.next(t0, t1, E)) {
      // this lane's token of a block: its row of X, loaded four blocks ahead (a block is copied faster than
      // a load comes back) and looked at when it is needed
      auto place_of = [&](int b) {
        const int r = b * kTok + q0 + static_cast<int>(lane & 7u);
        return r < w.n ? (job.index != nullptr ? job.index[w.lo + r] : w.lo + r) : -1;
      };
      constexpr int kAhead = 4;
      int ahead[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) ahead[k] = place_of(w.b0 + k);
      for (int b = w.b0; b < w.b1; ++b) {
        const int left = w.n - b * kTok;
        int place = ahead[0];
#pragma unroll
        for (int k = 0; k + 1 < kAhead; ++k) ahead[k] = ahead[k + 1];
        ahead[kAhead - 1] = place_of(b + kAhead);
        if (q0 + static_cast<int>(lane & 7u) < left && (place < 0 || place >= job.rows)) {
          if (a.status != nullptr && lane < 8 && f0 == 0) atomicOr(a.status, kDevBadIndex);
          place = -1;
        }
        ok = wait_all(bar_empty(stage), phase ^ 1u, abort_flag);
        if (!ok) break;
        if (!in_box(left)) {
          const uint32_t sx = sbase + stage * stage_bytes(RP) + part;
          const int rows = ((min(left, kTok) + 15) & ~15) - q0;  // those that the MMAs read
          if (rows > 0) {
#pragma unroll
            for (int p = 0; p < 8; ++p) {
              const int o = __shfl_sync(0xffffffffu, place, p);
              copy16(sx + swz(q0 + p, ch), x + static_cast<size_t>(max(o, 0)) * cols, there && o >= 0);
            }
          }
        }
        copy_arrive(bar_full(stage));
        if (++stage == S) stage = 0, phase ^= 1u;
      }
    }
    copy_wait<0>();
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    // adapters without rows, dealt out to the cluster's CTAs
    for (int e = rank; e < E; e += C) {
      if (s_off[e + 1] != s_off[e]) continue;
      const int wide = min(kWidth, cols - f0);
      for (int i = tid - 192; i < wide * (R / 8); i += 256) {
        const int row = i / (wide / 8);
        __nv_bfloat16* g = job.by_rank ? grad + (static_cast<size_t>(e) * R + row) * cols + f0 + (i - row * (wide / 8)) * 8
                                       : grad + (static_cast<size_t>(e) * cols + f0) * R + 8 * i;
        *reinterpret_cast<uint4*>(g) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  }

  // Stores four neighbouring ranks of feature f0 + f of adapter e.
  auto store4 = [&](int e, int f, int j, float4 v) {
    const int c = f0 + f;
    if (c >= cols || j >= R) return;
    const uint32_t p0 = pack_bf16(v.x, v.y), p1 = pack_bf16(v.z, v.w);
    if (job.by_rank) {
      __nv_bfloat16* g = grad + (static_cast<size_t>(e) * R + j) * cols + c;
      g[0] = __ushort_as_bfloat16(static_cast<unsigned short>(p0));
      g[cols] = __ushort_as_bfloat16(static_cast<unsigned short>(p0 >> 16));
      g[2 * static_cast<size_t>(cols)] = __ushort_as_bfloat16(static_cast<unsigned short>(p1));
      g[3 * static_cast<size_t>(cols)] = __ushort_as_bfloat16(static_cast<unsigned short>(p1 >> 16));
    } else {
      *reinterpret_cast<uint2*>(grad + (static_cast<size_t>(e) * cols + c) * R + j) = make_uint2(p0, p1);
    }
  };
  // Stores ranks j .. j + 15 of feature f0 + f of adapter e, f the lane's: neighbouring lanes exchange
  // halves, so that each has eight ranks of two features and a store touches half the lines.  (A backward
  // call of 64 rows of 32 adapters, rank 128, 4096 and 4096 features, took 88 us where each lane stored four
  // ranks of its own, 62 so.)
  auto store16 = [&](int e, int f, int j, const float (&v)[16]) {
    const bool odd = lane & 1u;
    uint32_t p[8], even_f[4], odd_f[4];
#pragma unroll
    for (int k = 0; k < 8; ++k) p[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? p[k] : p[k + 4], 1);
      even_f[k] = odd ? got : p[k];
      odd_f[k] = odd ? p[k + 4] : got;
    }
    const int c = f0 + (f & ~1);
    if (odd) j += 8;
    if (c >= cols || j >= R) return;
    if (job.by_rank) {
      uint32_t* g = reinterpret_cast<uint32_t*>(grad + (static_cast<size_t>(e) * R + j) * cols + c);
      const size_t step = static_cast<size_t>(cols) / 2;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        g[2 * k * step] = __byte_perm(even_f[k], odd_f[k], 0x5410);
        g[(2 * k + 1) * step] = __byte_perm(even_f[k], odd_f[k], 0x7632);
      }
    } else {
      uint4* g = reinterpret_cast<uint4*>(grad + (static_cast<size_t>(e) * cols + c) * R + j);
      g[0] = make_uint4(even_f[0], even_f[1], even_f[2], even_f[3]);
      g[R / 8] = make_uint4(odd_f[0], odd_f[1], odd_f[2], odd_f[3]);
    }
  };
  // The i-th of `per` features by RP / 4 fours of ranks, neighbours of those together that lie together.
  auto nth = [&](int i, int per, int& f, int& j4) {
    if (job.by_rank) {
      j4 = i / per;
      f = i - j4 * per;
    } else {
      f = i / 4 % per;
      j4 = i / (4 * per) * 4 + i % 4;
    }
  };
  // Partial sums of a CTA: those of the adapter that reaches in from the share before (0) and of the
  // one that reaches out into the next (1; before it, of long adapters within the share in turn),
  // [RP / 4][256 features] of four ranks.
  auto partial = [&](int p, int slot) {
    return reinterpret_cast<float4*>(a.partial) +
           ((static_cast<size_t>(blockIdx.x) / C * C + p) * 2 + slot) * (part_floats(RP) / 4);
  };
  if (warp >= 2 && warp < 6) {
    // ------------------------------------------------------------ epilogue
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    bool ok = true;
    int i = 0;
    while (ok && w.next(t0, t1, E)) {
      const bool whole = w.b0 == 0 && w.b1 == (w.n + kTok - 1) / kTok;
      float4* to = partial(rank, w.b0 > 0 ? 0 : 1);
      for (int c0 = w.b0; c0 < w.b1; c0 += kChain, ++i) {
        const int buf = bufs == 2 ? i & 1 : 0, use = bufs == 2 ? i >> 1 : i;
        ok = __all_sync(0xffffffffu, mbar_wait(bar_acc(buf), use & 1, abort_flag)) && !*abort_flag;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const bool store = whole && c0 + kChain >= w.b1;
        for (int h = 0; h < 2; ++h) {
          const int f = h * 128 + static_cast<int>(quarter * 32 + lane);
          for (int j = 0; j < RP; j += 16) {
            uint32_t x[16], y[16];
            const uint32_t ta = tmem + (quarter * 32u << 16) + buf * 4 * RP + h * 2 * RP + j;
            tmem_ld_x16(ta, x);
            tmem_ld_x16(ta + RP, y);
            float4 before[4];  // this thread's own sums of the runs before
            if (c0 != w.b0) {
#pragma unroll
              for (int q = 0; q < 4; ++q) before[q] = to[(j / 4 + q) * kWidth + f];
            }
            tmem_wait_ld();
            tmem_loaded(x);
            tmem_loaded(y);
            float v[16];
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = __uint_as_float(x[q]) + __uint_as_float(y[q]);
            if (c0 != w.b0) {
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                v[4 * q] += before[q].x, v[4 * q + 1] += before[q].y;
                v[4 * q + 2] += before[q].z, v[4 * q + 3] += before[q].w;
              }
            }
            if (store) {
              store16(w.e, f, j, v);
            } else {
#pragma unroll
              for (int q = 0; q < 4; ++q)
                to[(j / 4 + q) * kWidth + f] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_free(buf));
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
  }
  wait_for_launch_before();  // also where this CTA had no rows: the stream goes on behind this launch
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, tmem_cols);
  if (C == 1) return;
  __syncwarp();
  cluster_sync();  // every CTA's partial sums are in the workspace
  if (*abort_flag) return;
  Walk v = {s_off, -1, 0, 0, 0, 0, 0, 0};
  while (v.next(t0, t1, E)) {
    const int end = v.at + (v.n + kTok - 1) / kTok;
    if (v.at >= t0 && end <= t1) continue;
    // the CTAs with blocks of this adapter
    uint32_t with = 0;
    const float4* from[kMaxCluster];
    int p0 = 0;
#pragma unroll
    for (int p = 0; p < kMaxCluster; ++p) {
      if (p == C) break;
      const int p1 = share(blocks, p + 1, C);
      if (p0 < p1 && p0 < end && p1 > v.at) with |= 1u << p;
      from[p] = partial(p, v.at < p0 ? 0 : 1);
      p0 = p1;
    }
    const int count = __popc(with), k = __popc(with & ((1u << rank) - 1u));
    const int g0 = kWidth * k / count, per = kWidth * (k + 1) / count - g0;
    // Several sums at a time, each of up to eight CTAs' parts: their loads are what this takes.
    constexpr int kSums = 2;
    const int items = per * (RP / 4);
    for (int i0 = tid; i0 < items; i0 += kSums * kThreads) {
      float4 x[kSums][kMaxCluster];
      int f[kSums], j4[kSums];
#pragma unroll
      for (int q = 0; q < kSums; ++q) {
        const int i = min(i0 + q * kThreads, items - 1);
        nth(i, per, f[q], j4[q]);
        f[q] += g0;
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p)
          if ((with >> p) & 1u) x[q][p] = __ldcg(from[p] + j4[q] * kWidth + f[q]);
      }
#pragma unroll
      for (int q = 0; q < kSums; ++q) {
        float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int p = 0; p < kMaxCluster; ++p)
          if ((with >> p) & 1u) sum.x += x[q][p].x, sum.y += x[q][p].y, sum.z += x[q][p].z, sum.w += x[q][p].w;
        if (i0 + q * kThreads < items) store4(v.e, f[q], 4 * j4[q], sum);
      }
    }
  }
}

cudaError_t set_smem() {
  static thread_local uint64_t attr_ctx = 0;
  return set_smem_attr_once(reinterpret_cast<const void*>(lora_grad_kernel), 227 * 1024, &attr_ctx);
}

cudaLaunchConfig_t config(int cluster, long long items, size_t smem, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1] = dependent_launch();
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

// Clusters of c CTAs that the current context runs at once (none where it has a share of the SMs
// that is too small).  Asked once per context and thread.
int clusters_at_once(int c) {
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int active[kMaxCluster + 1];
  if (asked_ctx == 0 || asked_ctx != current_context_id()) {
    for (int k = 2; k <= kMaxCluster; ++k) {
      cudaLaunchAttribute attr[2] = {};
      const cudaLaunchConfig_t cfg = config(k, 1, 227 * 1024, attr);
      if (cudaOccupancyMaxActiveClusters(&active[k], lora_grad_kernel, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();  // a size that does not fit is no error of the call
        active[k] = 0;
      }
    }
    asked_ctx = current_context_id();
  }
  return active[c];
}

long long items_of(int cols) { return (static_cast<long long>(cols) + kWidth - 1) / kWidth; }

}  // namespace

size_t lora_q_bytes(int M, int E, int R) {
  const long long tiles = M / 128 + (M < E ? M : E);
  return static_cast<size_t>(tiles) * 2 * 256 * padded_rank(R);
}

size_t lora_partial_bytes(int M, int K, int N, int R) {
  // Clusters of several CTAs only where all CTAs together are at most kSms; a CTA by itself needs room where
  // an adapter's rows take several runs.
  const long long items = items_of(K) + items_of(N);
  long long ctas = 2 * items <= kSms ? kSms : 0;
  if (M > kChain * kTok && ctas < items) ctas = items;
  return sizeof(float) * static_cast<size_t>(ctas) * 2 * part_floats(padded_rank(R));
}

cudaError_t launch_lora_grad(LoraGradArgs a, cudaStream_t stream) {
  const cudaError_t err = set_smem();
  if (err != cudaSuccess) return err;
  const int RP = padded_rank(a.R);
  const long long items = items_of(a.job[0].cols) + items_of(a.job[1].cols);
  a.first1 = static_cast<int>(items_of(a.job[0].cols));
  a.stages = stages_of(RP);
  // As many CTAs to a feature block as run at once (15 clusters of eight, 36 of four) and as have two
  // token blocks each, or one adapter's: sums that several CTAs share cost as much as a block or two (512
  // rows of four adapters, rank 128, 2048 and 1536 features: 21 us by four CTAs, 28 by eight).
  const long long some = a.M < a.E ? a.M : a.E, pairs = (a.M / kTok + 1) / 2;
  const long long likely = pairs > some ? pairs : some;
  const int most = a.max_cluster > 0 && a.max_cluster < kMaxCluster ? a.max_cluster : kMaxCluster;
  int c = 1;
  for (int k = 2; k <= most; ++k)
    if (items * k <= kSms && k <= likely && items <= clusters_at_once(k)) c = k;
  a.cluster = c;
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t cfg =
      config(c, items, static_cast<size_t>(a.stages) * stage_bytes(RP) + misc_bytes(a.E), attr);
  cfg.stream = stream;
  if (a.M == 0) cfg.numAttrs = 1;  // no launch before has seen to it that the offsets are there
  return cudaLaunchKernelEx(&cfg, lora_grad_kernel, a);
}

}  // namespace mgw
