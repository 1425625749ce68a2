// Low-rank adapters of many requests at once beside a shared projection, and the data gradient:
//
//   u[r]   = x[t(r)] A[e]^T               v[r]  = dy[o(r)] B[e]
//   out[o] = base[o] + scale u[r] B[e]^T  dx[o] = dx_base[o] + scale v[r] A[e]
//
// Both are one kernel, `out = base + scale (in W1^T) W2^T` over a tile of 128 rows of one adapter:
// the data gradient reads B and A, as they are stored, in the other major order (TRANS).
//
// A cluster of up to eight CTAs takes a row tile.  Each contracts its share of the input's columns
// (tcgen05, 128 rows x rank, accumulators in TMEM), the CTAs' partial sums meet through distributed
// shared memory, a share of the rows each, and every CTA gets the tile's whole rank-wide
// intermediate as two bf16 parts (see split2) in its shared memory; from it each makes its share of
// the output's columns, 128 at a time.  So the intermediate never goes to HBM (but for u, where the
// backward pass wants it), one launch does it all, and few rows still use many SMs: a decode step's
// rows stream their adapters through eight SMs each.
//
// Roles (192 threads): warp 0 loads operands by TMA (x rows by gather4 where they are not a whole
// tile in order), warp 1 issues the MMAs, warps 2-5 hold the TMEM lane quarters: partial sums, then
// the output's epilogue (accumulator + base, rounded once, whole 128-byte row pieces).
#include <cuda_runtime.h>

#include <cstdint>

#include "lora.cuh"

namespace mgw {
namespace {

using namespace lora;

constexpr int kThreads = 192;
constexpr int kRows = 128;
constexpr int kBk = 64;               // input columns per stage
constexpr int kBn = 128;              // output columns per tile
constexpr int kXBytes = kRows * 128;  // 128 rows of 64 bf16
constexpr uint32_t kTmemCols = 256;   // two output tiles; the partial sums use the first one's
constexpr int kBars = 2 * 6 + 1 + 2 + 2 + 2 + 2 + 1;

// RB: 64-wide blocks of the rank.  The ring's memory is used again behind the contraction: partial
// sums (then the epilogue's staging), the intermediate's two parts, two tiles of W2.
template <int RB>
struct Plan {
  static constexpr int kStages = RB == 1 ? 4 : 6;
  static constexpr int kStage = kXBytes + RB * 8192;
  static constexpr int kPart = 0;
  static constexpr int kU = RB * 32768;
  static constexpr int kULo = kU + RB * kXBytes;
  static constexpr int kW2 = RB * 65536;
  static constexpr int kW2Tile = RB * 16384;
  static constexpr int kOffBar = RB * 98304;
  static constexpr int kOffTmp = kOffBar + kBars * 8;       // find_tile; [4] TMEM [5] abort
  static constexpr int kOffRows = (kOffTmp + 80 + 15) & ~15;  // place of the 128 output rows
  static constexpr size_t kSmem = kOffRows + kRows * 4 + 1024;
  static_assert(kStages * kStage <= kOffBar, "ring");
  static_assert(2 * kStages + 7 <= kBars, "barriers");
};
static_assert(2 * Plan<1>::kSmem <= 227 * 1024 && Plan<2>::kSmem <= 227 * 1024, "shared memory budget");

template <bool TRANS, int RB>
__global__ void __launch_bounds__(kThreads, RB == 1 ? 2 : 1) lora_kernel(const __grid_constant__ LoraArgs a) {
  using P = Plan<RB>;
  constexpr int S = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  int* s_tmp = reinterpret_cast<int*>(smem + P::kOffTmp);
  int* s_rows = reinterpret_cast<int*>(smem + P::kOffRows);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(s_tmp + 5);
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t lane = lane_id();
  const int C = a.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;

  RowTile t;
  if (!find_tile<kThreads, kRows>(a.off, a.E, a.M, static_cast<int>(blockIdx.x) / C, s_tmp, a.status, t)) return;
  if (t.nrows == 0) return;
  const int N = a.N;
  const int ntiles = (N + kBn - 1) / kBn;
  const int nt0 = static_cast<int>(static_cast<long long>(ntiles) * rank / C);
  const int nt1 = static_cast<int>(static_cast<long long>(ntiles) * (rank + 1) / C);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.base);

  if (t.e == a.E) {
    // Rows without an adapter: their base, or zeros.
    const int c0 = nt0 * kBn, c1 = min(nt1 * kBn, N);
    for (int i = warp; i < t.nrows; i += kThreads / 32) {
      const int r = t.row0 + i;
      if (a.u != nullptr && rank == 0)
        for (int j = static_cast<int>(lane); j < a.R; j += 32) a.u[static_cast<size_t>(r) * a.R + j] = 0.0f;
      if (out == nullptr || out == base) continue;
      const int o = row_place(a.out_index, r, a.out_rows, lane == 0 ? a.status : nullptr);
      if (o < 0) continue;
      for (int c = c0 + static_cast<int>(lane) * 8; c < c1; c += 256) {
        const size_t at = static_cast<size_t>(o) * N + c;
        uint4 v = make_uint4(0u, 0u, 0u, 0u);
        if (base != nullptr) v = *reinterpret_cast<const uint4*>(base + at);
        *reinterpret_cast<uint4*>(out + at) = v;
      }
    }
    return;
  }

  const uint32_t bar0 = sbase + P::kOffBar;
  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (S + s); };
  const uint32_t bar_sum = bar0 + 8u * (2 * S);
  auto bar_wfull = [&](int s) { return bar0 + 8u * (2 * S + 1 + s); };
  auto bar_wempty = [&](int s) { return bar0 + 8u * (2 * S + 3 + s); };
  auto bar_acc = [&](int s) { return bar0 + 8u * (2 * S + 5 + s); };
  auto bar_free = [&](int s) { return bar0 + 8u * (2 * S + 7 + s); };
  const uint32_t bar_done = bar0 + 8u * (2 * S + 9);
  if (tid == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar_full(s), 1);
      mbar_init(bar_empty(s), 1);
    }
    mbar_init(bar_sum, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_wfull(s), 1);
      mbar_init(bar_wempty(s), 1);
      mbar_init(bar_acc(s), 1);
      mbar_init(bar_free(s), 4);
    }
    mbar_init(bar_done, 1);
    fence_mbar_init();
    s_tmp[5] = 0;
    tma_prefetch_desc(&a.tm_w1);
    tma_prefetch_desc(&a.tm_w2);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmp + 4), kTmemCols);
    tmem_relinquish();
  }
  if (tid >= 64) {
    const int i = tid - 64;
    s_rows[i] = i < t.nrows ? row_place(a.out_index, t.row0 + i, a.out_rows, rank == 0 ? a.status : nullptr) : -1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_tmp[4]);
  const int RP = (a.R + 15) & ~15;
  const int nch = (a.K + kBk - 1) / kBk;
  const int c0 = static_cast<int>(static_cast<long long>(nch) * rank / C);
  const int c1 = static_cast<int>(static_cast<long long>(nch) * (rank + 1) / C);

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    const bool whole = a.in_index == nullptr && t.nrows == kRows;
    int idx[4];
    const int groups = (t.nrows + 3) >> 2;
    if (!whole) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * static_cast<int>(lane) + j;
        idx[j] = i < t.nrows ? row_place(a.in_index, t.row0 + i, a.in_rows, rank == 0 ? a.status : nullptr) : -1;
      }
    }
    const uint32_t w1_bytes = TRANS ? RB * 8192u : static_cast<uint32_t>(RP) * 128u;
    const uint32_t x_bytes = whole ? static_cast<uint32_t>(kXBytes) : static_cast<uint32_t>(groups) * 512u;
    bool ok = true;
    int stage = 0, n = 0;
    uint32_t phase = 0;
    for (int c = c0; c < c1; ++c) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_empty(stage), phase ^ 1u, abort_flag))) {
        ok = false;
        break;
      }
      const uint32_t fb = bar_full(stage);
      const uint32_t sx = sbase + stage * P::kStage, sw = sx + kXBytes;
      if (lane == 0) {
        mbar_arrive_expect_tx(fb, x_bytes + w1_bytes);
        if constexpr (TRANS) {
#pragma unroll
          for (int b = 0; b < RB; ++b) tma_load_3d(sw + b * 8192, &a.tm_w1, 64 * b, c * kBk, t.e, fb);
        } else {
          tma_load_3d(sw, &a.tm_w1, c * kBk, 0, t.e, fb);
        }
        if (whole) tma_load_2d(sx, &a.tm_x, c * kBk, t.row0, fb);
      }
      __syncwarp();
      if (!whole && static_cast<int>(lane) < groups) tma_gather4(sx + lane * 512u, &a.tm_xg, c * kBk, idx, fb);
      ++n;
      if (++stage == S) stage = 0, phase ^= 1u;
    }
    // W2 lies in the ring's memory: behind the last MMA that reads the ring.
    ok = __all_sync(0xffffffffu, ok && mbar_wait(bar_sum, 0, abort_flag));
    int w = 0;
    auto load_w2 = [&](int nt) {
      const uint32_t fb = bar_wfull(w & 1), dst = sbase + P::kW2 + (w & 1) * P::kW2Tile;
      if (lane == 0) {
        if constexpr (TRANS) {
          mbar_arrive_expect_tx(fb, 2u * RP * 128u);
          tma_load_3d(dst, &a.tm_w2, nt * kBn, 0, t.e, fb);
          tma_load_3d(dst + P::kW2Tile / 2, &a.tm_w2, nt * kBn + 64, 0, t.e, fb);
        } else {
          mbar_arrive_expect_tx(fb, P::kW2Tile);
#pragma unroll
          for (int b = 0; b < RB; ++b) tma_load_3d(dst + b * 16384, &a.tm_w2, 64 * b, nt * kBn, t.e, fb);
        }
      }
      ++w;
    };
    int nt = nt0;
    if (ok && out != nullptr)
      for (; nt < nt1 && w < 2; ++nt) load_w2(nt);
    __syncwarp();
    cluster_sync();  // partial sums are there
    cluster_sync();  // the intermediate is
    for (; ok && out != nullptr && nt < nt1; ++nt) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar_wempty(w & 1), ((w >> 1) & 1) ^ 1u, abort_flag));
      if (ok) load_w2(nt);
      __syncwarp();
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    // Never leave the CTA with copies still landing in shared memory.
    for (int i = n > S ? n - S : 0; i < n; ++i) mbar_wait_drain(bar_full(i % S), (i / S) & 1u);
    for (int i = w > 2 ? w - 2 : 0; i < w; ++i) mbar_wait_drain(bar_wfull(i & 1), (i >> 1) & 1u);
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const bool issue = elect_one();
    bool ok = true;
    {
      const uint32_t idesc = idesc_bf16(RP, false, TRANS);
      int stage = 0;
      uint32_t phase = 0;
      for (int c = c0; c < c1; ++c) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_full(stage), phase, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sx = sbase + stage * P::kStage, sw = sx + kXBytes;
        const uint64_t ad = sdesc_kmajor_sw128(sx);
        const uint64_t bd = TRANS ? sdesc_mn_sw128(sw, 8192) : sdesc_kmajor_sw128(sw);
        if (issue) {
#pragma unroll
          for (uint32_t k = 0; k < kBk / 16; ++k)
            mma_bf16(tmem, ad + kStepK * k, bd + (TRANS ? kStepMn : kStepK) * k, idesc, c != c0 || k != 0);
          mma_commit(bar_empty(stage));
        }
        __syncwarp();
        if (++stage == S) stage = 0, phase ^= 1u;
      }
      if (issue) mma_commit(bar_sum);
      __syncwarp();
    }
    cluster_sync();
    cluster_sync();
    tc_fence_after();
    fence_async_all();
    if (out != nullptr) {
      const uint32_t idesc = idesc_bf16(kBn, false, TRANS);
      for (int nt = nt0, i = 0; ok && nt < nt1; ++nt, ++i) {
        const int s = i & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(bar_wfull(s), (i >> 1) & 1, abort_flag) &&
                                         mbar_wait(bar_free(s), ((i >> 1) & 1) ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sw = sbase + P::kW2 + s * P::kW2Tile;
        const uint32_t d = tmem + static_cast<uint32_t>(s * kBn);
        if (issue) {
          for (int part = 0; part < 2; ++part) {
            for (int k = 0; k < RP / 16; ++k) {
              // 16 ranks: 32 bytes within a 64-wide block of the intermediate
              const uint32_t su = sbase + (part ? P::kULo : P::kU) + (k >> 2) * kXBytes;
              const uint64_t ad = sdesc_kmajor_sw128(su) + kStepK * (k & 3);
              const uint64_t bd = TRANS ? sdesc_mn_sw128(sw, P::kW2Tile / 2) + kStepMn * k
                                        : sdesc_kmajor_sw128(sw + (k >> 2) * 16384) + kStepK * (k & 3);
              mma_bf16(d, ad, bd, idesc, part != 0 || k != 0);
            }
          }
          mma_commit(bar_wempty(s));
          mma_commit(bar_acc(s));
        }
        __syncwarp();
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
    if (issue) {
      mma_commit(bar_done);
      mbar_wait_drain(bar_done, 0);
    }
    __syncwarp();
  } else {
    // ------------------------------------------- partial sums, then the epilogue
    const int quarter = warp & 3;
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const uint32_t part = sbase + P::kPart;
    bool ok = __all_sync(0xffffffffu, mbar_wait(bar_sum, 0, abort_flag));
    tc_fence_after();
    // Partial sums as [RP / 4][128 rows] of four ranks: a warp's 32 rows lie side by side.
    if (ok) {
      const uint32_t row = static_cast<uint32_t>(quarter * 32) + lane;
      for (int j = 0; j < RP; j += 16) {
        uint32_t r[16];
        tmem_ld_x16(tq + j, r);
        tmem_wait_ld();
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_shared_f4(part + ((j / 4 + q) * kRows + row) * 16u, __uint_as_float(r[4 * q]),
                       __uint_as_float(r[4 * q + 1]), __uint_as_float(r[4 * q + 2]),
                       __uint_as_float(r[4 * q + 3]));
      }
    }
    tc_fence_before();
    __syncwarp();
    cluster_sync();
    {
      // This CTA's rows of the tile: summed over the CTAs in their order, eight ranks at a time.
      const float scale = a.scale != nullptr ? a.scale[t.e] : 1.0f;
      const int per = kRows / C, r0 = rank * per;
      for (int i = tid - 64; i < per * (RP / 8); i += 128) {
        const int row = r0 + i % per, j8 = i / per;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        if (row < t.nrows && 8 * j8 < a.R) {
          const uint32_t at = part + (2u * j8 * kRows + row) * 16u;
          for (int p = 0; p < C; ++p) {
            const uint32_t from = map_to_cta(at, p);
            const float4 x = ld_cluster_f4(from), y = ld_cluster_f4(from + kRows * 16u);
            v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
            v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
          }
          if (a.u != nullptr) {
            float4* u = reinterpret_cast<float4*>(a.u + static_cast<size_t>(t.row0 + row) * a.R + 8 * j8);
            u[0] = make_float4(v[0], v[1], v[2], v[3]);
            u[1] = make_float4(v[4], v[5], v[6], v[7]);
          }
        }
        uint4 hi, lo;
        split2(v[0] * scale, v[1] * scale, hi.x, lo.x);
        split2(v[2] * scale, v[3] * scale, hi.y, lo.y);
        split2(v[4] * scale, v[5] * scale, hi.z, lo.z);
        split2(v[6] * scale, v[7] * scale, hi.w, lo.w);
        const uint32_t to = sbase + P::kU + (j8 >> 3) * kXBytes + swz(row, j8 & 7);
        for (int p = 0; p < C; ++p) {
          const uint32_t dst = map_to_cta(to, p);
          st_cluster_u4(dst, hi);
          st_cluster_u4(dst + RB * kXBytes, lo);
        }
      }
    }
    fence_async_all();
    __syncwarp();
    cluster_sync();
    if (out != nullptr) {
      // Half a tile (64 columns) at a time: fp32 sums into this warp's staging (32 rows of 16 chunks
      // of 16 bytes, chunk c of row r at c ^ (r & 7)), and out again as whole row pieces, eight lanes
      // to a row.
      const uint32_t stage = sbase + P::kPart + static_cast<uint32_t>(warp - 2) * 8192u;
      const int sub = static_cast<int>(lane >> 3), ch = static_cast<int>(lane & 7);
      int place[8];
#pragma unroll
      for (int p = 0; p < 8; ++p) place[p] = s_rows[quarter * 32 + 4 * p + sub];
      const uint32_t odd = static_cast<uint32_t>(ch >> 2);
      for (int nt = nt0, i = 0; nt < nt1; ++nt, ++i) {
        const int s = i & 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int col = nt * kBn + 64 * h + 8 * ch;
          uint4 bv[8];
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            bv[p] = make_uint4(0u, 0u, 0u, 0u);
            if (base != nullptr && place[p] >= 0 && col < N)
              bv[p] = *reinterpret_cast<const uint4*>(base + static_cast<size_t>(place[p]) * N + col);
          }
          if (h == 0) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait(bar_acc(s), (i >> 1) & 1, abort_flag));
            tc_fence_after();
          }
          if (!ok) break;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t r[32];
            tmem_ld_32x32b_x32(tq + s * kBn + 64 * h + 32 * q, r);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 8; ++c)
              st_shared_f4(stage + lane * 256u + (((8u * q + c) ^ (lane & 7u)) << 4), __uint_as_float(r[4 * c]),
                           __uint_as_float(r[4 * c + 1]), __uint_as_float(r[4 * c + 2]),
                           __uint_as_float(r[4 * c + 3]));
          }
          if (h == 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_free(s));
          }
          __syncwarp();
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const uint32_t r = 4u * p + sub, at = stage + r * 256u;
            // lanes 4 .. 7 of a row read their second chunk first: eight different bank groups
            float4 f[2];
            f[0] = ld_shared_f4(at + (((2u * ch + odd) ^ (r & 7u)) << 4));
            f[1] = ld_shared_f4(at + (((2u * ch + 1u - odd) ^ (r & 7u)) << 4));
            const float4 x = odd ? f[1] : f[0], y = odd ? f[0] : f[1];
            const float2 b0 = unpack_bf16(bv[p].x), b1 = unpack_bf16(bv[p].y), b2 = unpack_bf16(bv[p].z),
                         b3 = unpack_bf16(bv[p].w);
            uint4 v;
            v.x = pack_bf16(b0.x + x.x, b0.y + x.y);
            v.y = pack_bf16(b1.x + x.z, b1.y + x.w);
            v.z = pack_bf16(b2.x + y.x, b2.y + y.y);
            v.w = pack_bf16(b3.x + y.z, b3.y + y.w);
            if (place[p] >= 0 && col < N)
              *reinterpret_cast<uint4*>(out + static_cast<size_t>(place[p]) * N + col) = v;
          }
          __syncwarp();
        }
        if (!ok) break;
      }
    }
    if (!ok && lane == 0) {
      *abort_flag = 1;
      if (a.status) atomicOr(a.status, kDevTimeout);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <bool TRANS, int RB>
cudaError_t set_smem() {
  static thread_local uint64_t attr_ctx = 0;
  return set_smem_attr_once(reinterpret_cast<const void*>(lora_kernel<TRANS, RB>), Plan<RB>::kSmem, &attr_ctx);
}

template <bool TRANS, int RB>
cudaLaunchConfig_t config(int cluster, long long tiles, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Plan<RB>::kSmem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = static_cast<unsigned>(cluster);
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

// The largest cluster, up to eight CTAs, that the current context can run (a share of the SMs may be
// too small for it).  Asked once per context and thread.
template <bool TRANS, int RB>
int largest_cluster() {
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int largest = 1;
  if (asked_ctx != 0 && asked_ctx == current_context_id()) return largest;
  largest = 1;
  for (int c = 8; c > 1; c /= 2) {
    cudaLaunchAttribute attr = {};
    const cudaLaunchConfig_t cfg = config<TRANS, RB>(c, 1, &attr);
    int active = 0;
    if (cudaOccupancyMaxActiveClusters(&active, lora_kernel<TRANS, RB>, &cfg) != cudaSuccess) {
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

template <bool TRANS, int RB>
cudaError_t launch(LoraArgs a, int num_sms, cudaStream_t stream) {
  cudaError_t err = set_smem<TRANS, RB>();
  if (err != cudaSuccess) return err;
  // The exact number of tiles is known on the device only: at most this many, the tiles of rows
  // without an adapter included.
  const long long some = a.M < a.E ? a.M : a.E;
  const long long tiles = a.M / kRows + some + 1;
  // As many CTAs to a tile as the SMs have room for; each needs some columns of its own.
  const long long expected = (a.M + kRows - 1) / kRows + some / 2;
  const int nch = (a.K + kBk - 1) / kBk;
  int most = largest_cluster<TRANS, RB>();
  if (a.max_cluster > 0 && a.max_cluster < most) most = a.max_cluster;
  int c = 1;
  while (2 * c <= most && 2 * c <= nch && expected * 2 * c <= num_sms * (RB == 1 ? 2 : 1)) c *= 2;
  a.cluster = c;
  cudaLaunchAttribute attr = {};
  cudaLaunchConfig_t cfg = config<TRANS, RB>(c, tiles, &attr);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, lora_kernel<TRANS, RB>, a);
}

}  // namespace

cudaError_t launch_lora(const LoraArgs& a, bool transposed, int num_sms, cudaStream_t stream) {
  if (a.R > 64)
    return transposed ? launch<true, 2>(a, num_sms, stream) : launch<false, 2>(a, num_sms, stream);
  return transposed ? launch<true, 1>(a, num_sms, stream) : launch<false, 1>(a, num_sms, stream);
}

}  // namespace mgw
