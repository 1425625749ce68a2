// Gradients of the low-rank adapters: for the rows r of adapter e
//
//   dA[e][j][k] = scale[e] sum_r v[r][j] x[t(r)][k]      dB[e][n][j] = scale[e] sum_r dy[o(r)][n] u[r][j]
//
// Both are grad = X^T Q, X bf16 rows contracted over the rows (as the weight gradient of an expert),
// Q fp32 [M, R] rank-wide.  X's rows arrive as they lie in memory, 64 tokens by 64 features, and
// the tensor core reads them across (MN-major, see lora.cuh): nothing is transposed.  Q is split into
// two bf16 parts (split2) on the way, both in one product of twice the rank's width.
//
// A work item is (adapter, 128 or 256 features); a cluster of up to eight CTAs shares its rows and
// adds up its fp32 sums, in the CTAs' order, through distributed shared memory: no atomics and no
// workspace, the same bits on every run.
//
// Roles (192 threads): warp 0 loads by TMA, warp 1 issues the MMAs, warps 2-5 split Q (a thread a
// rank and eight tokens: reads along the ranks, writes 16 bytes of one rank's tokens), then store.
#include <cuda_runtime.h>

#include <cstdint>

#include "lora.cuh"

namespace mgw {
namespace {

using namespace lora;

constexpr int kThreads = 192;
constexpr int kTok = 64;  // tokens per stage
constexpr int kMaxStages = 6;
constexpr int kMiscBytes = 8 * (3 * kMaxStages + 2) + 16 + 1024;

struct Shape {
  int fb, stages, stage_bytes;
  uint32_t tmem_cols;
  size_t smem;
};
__host__ __device__ constexpr int padded_rank(int R) { return (R + 15) & ~15; }
__host__ __device__ constexpr int feature_blocks(int R) { return padded_rank(R) <= 32 ? 1 : 2; }
__host__ __device__ constexpr Shape shape_of(int R) {
  const int rp = padded_rank(R);
  Shape s = {};
  s.fb = feature_blocks(R);
  s.stage_bytes = s.fb * 16384 + 2 * rp * 256;  // X, Q in fp32, its two parts
  // two CTAs an SM up to rank 32, one beyond (deep enough rings do not fit twice)
  const int room = (s.fb == 1 ? 113 : 226) * 1024 - kMiscBytes;
  s.stages = room / s.stage_bytes < kMaxStages ? room / s.stage_bytes : kMaxStages;
  s.tmem_cols = 32;
  while (s.tmem_cols < static_cast<uint32_t>(s.fb * 2 * rp)) s.tmem_cols *= 2;
  s.smem = static_cast<size_t>(s.stages) * s.stage_bytes + kMiscBytes;
  return s;
}
static_assert(shape_of(16).stages >= 3 && shape_of(32).stages >= 3 && shape_of(64).stages >= 3 &&
                  shape_of(128).stages >= 2 && shape_of(128).tmem_cols <= 512,
              "ring");
// the CTA's fp32 sums lie in the ring at the end
static_assert(128 * 2 * 128 * 4 <= shape_of(128).stages * shape_of(128).stage_bytes &&
                  128 * 2 * 48 * 4 <= shape_of(48).stages * shape_of(48).stage_bytes,
              "sums");

template <int FB>
__global__ void __launch_bounds__(kThreads, FB == 1 ? 2 : 1) lora_grad_kernel(const __grid_constant__ LoraGradArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t lane = lane_id();
  const int C = a.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int R = a.R, RP = padded_rank(R);
  const int S = a.stages, stage_bytes = FB * 16384 + 2 * RP * 256;
  const uint32_t raw_at = FB * 16384, part_at = raw_at + RP * 256;
  uint8_t* misc = smem + S * stage_bytes;
  int* s_misc = reinterpret_cast<int*>(misc + 8 * (3 * kMaxStages + 2));  // [0] TMEM [1] abort
  volatile int* abort_flag = reinterpret_cast<volatile int*>(s_misc + 1);

  int bad = 0;
  for (int i = tid; i < a.E; i += kThreads) bad |= a.off[i + 1] < a.off[i];
  if (tid == 0) bad |= a.off[0] != 0 || a.off[a.E] > a.M;
  if (__syncthreads_or(bad)) {
    if (tid == 0 && a.status != nullptr) atomicOr(a.status, kDevBadOffsets);
    return;
  }
  int item = static_cast<int>(blockIdx.x) / C;
  const int which = item >= a.first[1] ? 1 : 0;
  item -= a.first[which];
  const LoraGradJob& job = a.job[which];
  const int width = FB * 128;
  const int blocks = (job.cols + width - 1) / width;
  const int e = item / blocks, f0 = item % blocks * width;
  const int lo = a.off[e], n = a.off[e + 1] - lo;
  const int cols = job.cols;
  __nv_bfloat16* grad = static_cast<__nv_bfloat16*>(job.grad);

  // Stores four neighbouring ranks of feature f0 + f.
  auto store4 = [&](int f, int j, float4 v) {
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
  const int per = width / C;  // features that this CTA stores
  if (n == 0) {
    for (int i = tid; i < per * (RP / 4); i += kThreads)
      store4(rank * per + i % per, i / per * 4, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    return;
  }
  const int tiles = (n + kTok - 1) / kTok;
  const int t0 = static_cast<int>(static_cast<long long>(tiles) * rank / C);
  const int t1 = static_cast<int>(static_cast<long long>(tiles) * (rank + 1) / C);

  const uint32_t bar0 = smem_u32(misc);
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto bar_part = [&](int s) { return bar0 + 8u * (2 * kMaxStages + s); };
  const uint32_t bar_acc = bar0 + 8u * (3 * kMaxStages);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
      mbar_init(bar_part(s), 4);
    }
    mbar_init(bar_acc, 1);
    fence_mbar_init();
    s_misc[1] = 0;
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_misc), a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_misc[0]);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const int l = static_cast<int>(lane & 15u);
    bool ok = true;
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    int idx[4];
    auto load_idx = [&](int t) {
      if (job.index == nullptr) return;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = t * kTok + 4 * l + j;
        idx[j] = t < t1 && i < n ? job.index[lo + i] : -1;
      }
    };
    load_idx(t0);
    for (int t = t0; t < t1; ++t) {
      const int valid = min(kTok, n - t * kTok);
      const int groups = ((valid + 15) & ~15) >> 2;  // the tokens that the MMAs read
      const bool whole = job.index == nullptr && valid == kTok;
      int r[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * l + j;
        r[j] = -1;
        if (i < valid) {
          r[j] = job.index == nullptr ? lo + t * kTok + i : idx[j];
          if (r[j] < 0 || r[j] >= job.rows) {
            if (a.status != nullptr) atomicOr(a.status, kDevBadIndex);
            r[j] = -1;
          }
        }
      }
      load_idx(t + 1);
      if (!__all_sync(0xffffffffu, mbar_wait(bar_empty(stage), phase ^ 1u, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t fb = bar_full(stage), sx = sbase + stage * stage_bytes;
      if (lane == 0) {
        const uint32_t q_bytes = static_cast<uint32_t>(valid * R) * 4u;
        mbar_arrive_expect_tx(fb, (whole ? FB * 16384u : static_cast<uint32_t>(groups) * 512u * 2 * FB) + q_bytes);
        bulk_load(sx + raw_at, job.q + static_cast<size_t>(lo + t * kTok) * R, q_bytes, fb);
        if (whole) {
#pragma unroll
          for (int b = 0; b < 2 * FB; ++b)
            tma_load_2d(sx + b * 8192, &job.tm, f0 + 64 * b, lo + t * kTok, fb);
        }
      }
      __syncwarp();
      if (!whole && l < groups) {
#pragma unroll
        for (int b = 0; b < FB; ++b) {
          const int at = 2 * b + static_cast<int>(lane >> 4);
          tma_gather4(sx + at * 8192 + l * 512, &job.tmg, f0 + 64 * at, r, fb);
        }
      }
      ++filled;
      if (++stage == S) stage = 0, phase ^= 1u;
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
    int stage = 0;
    uint32_t phase = 0;
    for (int t = t0; t < t1; ++t) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_full(stage), phase, abort_flag) &&
                                       mbar_wait(bar_part(stage), phase, abort_flag))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t sx = sbase + stage * stage_bytes;
      const int steps = (min(kTok, n - t * kTok) + 15) >> 4;
      if (issue) {
        const uint64_t bd = sdesc_kmajor_sw128(sx + part_at);
#pragma unroll
        for (int b = 0; b < FB; ++b) {
          const uint64_t ad = sdesc_mn_sw128(sx + b * 16384, 8192);
          for (int k = 0; k < steps; ++k)
            mma_bf16(tmem + b * 2 * RP, ad + kStepMn * k, bd + kStepK * k, idesc, t != t0 || k != 0);
        }
        mma_commit(bar_empty(stage));
      }
      __syncwarp();
      if (++stage == S) stage = 0, phase ^= 1u;
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    if (issue) {
      mma_commit(bar_acc);
      mbar_wait_drain(bar_acc, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------- Q's two parts, then the sums
    const float scale = a.scale != nullptr ? a.scale[e] : 1.0f;
    const int ct = tid - 64;  // 0 .. 127
    bool ok = true;
    int stage = 0;
    uint32_t phase = 0;
    for (int t = t0; t < t1; ++t) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_full(stage), phase, abort_flag))) {
        ok = false;
        break;
      }
      const int valid = min(kTok, n - t * kTok);
      const uint32_t sx = sbase + stage * stage_bytes;
      for (int i = ct; i < RP * 8; i += 128) {
        const int j = i % RP, o = i / RP;  // rank, eight tokens
        float v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int tok = 8 * o + k;
          v[k] = j < R && tok < valid ? scale * ld_shared_f1(sx + raw_at + static_cast<uint32_t>(tok * R + j) * 4u) : 0.0f;
        }
        uint4 hi, lo4;
        split2(v[0], v[1], hi.x, lo4.x);
        split2(v[2], v[3], hi.y, lo4.y);
        split2(v[4], v[5], hi.z, lo4.z);
        split2(v[6], v[7], hi.w, lo4.w);
        const uint32_t at = sx + part_at + swz(j, o);
        st_shared_u4(at, hi);
        st_shared_u4(at + RP * 128, lo4);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_part(stage));
      if (++stage == S) stage = 0, phase ^= 1u;
    }
    ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_acc, 0, abort_flag));
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    tc_fence_after();
    // this CTA's sums as [RP / 4][width] of four ranks
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    for (int b = 0; b < FB; ++b) {
      const uint32_t f = b * 128u + quarter * 32u + lane;
      for (int j = 0; j < RP; j += 16) {
        uint32_t h[16], l[16];
        if (t1 > t0 && ok) {
          const uint32_t ta = tmem + (quarter * 32u << 16) + b * 2 * RP + j;
          tmem_ld_x16(ta, h);
          tmem_ld_x16(ta + RP, l);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) h[k] = l[k] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_shared_f4(sbase + (static_cast<uint32_t>((j / 4 + q) * width) + f) * 16u,
                       __uint_as_float(h[4 * q]) + __uint_as_float(l[4 * q]),
                       __uint_as_float(h[4 * q + 1]) + __uint_as_float(l[4 * q + 1]),
                       __uint_as_float(h[4 * q + 2]) + __uint_as_float(l[4 * q + 2]),
                       __uint_as_float(h[4 * q + 3]) + __uint_as_float(l[4 * q + 3]));
      }
    }
    tc_fence_before();
    __syncwarp();
  }
  __syncthreads();
  cluster_sync();  // every CTA's sums are there
  if (!*abort_flag) {
    for (int i = tid; i < per * (RP / 4); i += kThreads) {
      const int f = rank * per + i % per, j4 = i / per;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int p = 0; p < C; ++p) {
        const float4 x = ld_cluster_f4(map_to_cta(sbase + static_cast<uint32_t>(j4 * width + f) * 16u, p));
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      store4(f, 4 * j4, v);
    }
  }
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, a.tmem_cols);
  __syncwarp();
  cluster_sync();  // nobody reads this CTA's sums any more
}

template <int FB>
cudaError_t set_smem() {
  static thread_local uint64_t attr_ctx = 0;
  return set_smem_attr_once(reinterpret_cast<const void*>(lora_grad_kernel<FB>), 227 * 1024, &attr_ctx);
}

template <int FB>
cudaLaunchConfig_t config(int cluster, long long items, size_t smem, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(items * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(cluster);
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// The largest cluster, up to eight CTAs, that the current context can run; asked once per context
// and thread, for the largest shared memory.
template <int FB>
int largest_cluster() {
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int largest = 1;
  if (asked_ctx != 0 && asked_ctx == current_context_id()) return largest;
  largest = 1;
  for (int c = 8; c > 1; c /= 2) {
    cudaLaunchAttribute attr = {};
    const cudaLaunchConfig_t cfg = config<FB>(c, 1, 226 * 1024, &attr);
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, lora_grad_kernel<FB>, &cfg) != cudaSuccess) {
      (void)cudaGetLastError();  // a size that does not fit is no error of the call
      active = 0;
    }
    if (active > 0) {
      largest = c;
      break;
    }
  }
  asked_ctx = current_context_id();
  return largest;
}

template <int FB>
cudaError_t launch(LoraGradArgs a, int num_sms, cudaStream_t stream) {
  const cudaError_t err = set_smem<FB>();
  if (err != cudaSuccess) return err;
  const Shape s = shape_of(a.R);
  long long items[2] = {0, 0};
  for (int i = 0; i < a.jobs; ++i)
    items[i] = static_cast<long long>(a.E) * ((a.job[i].cols + FB * 128 - 1) / (FB * 128));
  a.first[0] = 0;
  a.first[1] = a.jobs == 2 ? static_cast<int>(items[0]) : 0x7fffffff;
  a.stages = s.stages;
  a.tmem_cols = s.tmem_cols;
  int most = largest_cluster<FB>();
  if (a.max_cluster > 0 && a.max_cluster < most) most = a.max_cluster;
  const long long total = items[0] + items[1];
  int c = 1;
  while (2 * c <= most && 2 * c * kTok <= a.M && total * 2 * c <= num_sms * (FB == 1 ? 2 : 1)) c *= 2;
  a.cluster = c;
  cudaLaunchAttribute attr = {};
  cudaLaunchConfig_t cfg = config<FB>(c, total, s.smem, &attr);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, lora_grad_kernel<FB>, a);
}

}  // namespace

long long lora_grad_items(int E, int cols, int R) {
  const int width = feature_blocks(R) * 128;
  return static_cast<long long>(E) * ((cols + width - 1) / width);
}

cudaError_t launch_lora_grad(const LoraGradArgs& a, int num_sms, cudaStream_t stream) {
  return feature_blocks(a.R) == 1 ? launch<1>(a, num_sms, stream) : launch<2>(a, num_sms, stream);
}

}  // namespace mgw
