// Low-rank adapters for few rows, a decode step's: out[o] = base[o] + scale (x[t] A[e]^T) B[e]^T.
//
// With a row or a few to an adapter the call is a read of the adapters, and below a few MB it is
// latency: of the launch, of loads that wait for loads.  So a cluster of CTAs takes up to eight rows of
// one adapter, each CTA some columns of x and A, then some of out, and every load is made as early as its
// address is known: B's and base's first pieces before the CTAs exchange their sums.
//
// The products run on mma.sync m16n8k16 with the adapter as the 16-row operand and the rows of x as the
// eight columns: its operands come straight from global memory into registers, 16 bytes a lane.  (Which
// of the contraction's columns a register stands for is the caller's choice as long as both operands
// agree, so a lane's 16 bytes are two steps' worth.)  Through tcgen05 the same rows take operand
// tiles in shared memory, TMEM and four more waits: 16 rows of 16 adapters, rank 16, 4096 x 4096, take
// lora.cu's kernel 19 us and this one 6, which is launch and four loads that wait for one another
// (offsets, row index, x and A, the other CTAs' sums).  128 rows of 32 adapters, rank 64, 4096 x 8192: 17 us
// for 55 MB.  B's first pieces are in registers while A's sums are exchanged, which takes all 128 that two CTAs
// an SM have: the build for rank 33 to 64 spills 36 bytes a thread, that for more 12.
#include <cuda_runtime.h>

#include <cstdint>

#include "lora.cuh"

namespace mgw {
namespace {

using namespace lora;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;  // rows of a tile: the products' N
constexpr int kMaxCluster = 8;

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9},"
      " {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 32 of the contraction: a lane's 16 bytes of rows g and g + 8, and of the column's.
__device__ __forceinline__ void mma_32(float (&c)[4], uint4 top, uint4 bottom, uint4 b) {
  mma_16816(c, top.x, bottom.x, top.y, bottom.y, b.x, b.y);
  mma_16816(c, top.z, bottom.z, top.w, bottom.w, b.z, b.w);
}
__device__ __forceinline__ uint4 load16(const __nv_bfloat16* p, bool there) {
  return there ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0u, 0u, 0u, 0u);
}
__device__ __forceinline__ void st_cluster_f1(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// NB: 32-wide blocks of the rank.
template <int NB>
struct Few {
  static constexpr int kRanks = 32 * NB;
  static constexpr int kTiles = NB == 4 ? 2 : 4;  // 16-wide tiles of out's columns a warp takes at once
  static constexpr int kCols = 16 * kTiles;
  static constexpr int kPitch = kRanks + 8;       // of the intermediate's rows: no bank conflicts
  static constexpr int kSums = kRanks * kRows;
  static constexpr int kTurn = kWarps * kRows * (kCols + 4);
  static constexpr int kOffU = 4 * (kMaxCluster * kSums + (kWarps * kSums > kTurn ? kWarps * kSums : kTurn));
  static constexpr size_t kSmem = kOffU + 2 * kRows * kPitch * 2;
  static_assert(kOffU % 16 == 0 && kPitch % 8 == 0 && (kCols + 4) % 4 == 0, "alignment");
};

template <int NB>
__global__ void __launch_bounds__(kThreads, 2) lora_few_kernel(const LoraArgs a) {
  using F = Few<NB>;
  extern __shared__ __align__(16) uint8_t smem[];
  float* s_cta = reinterpret_cast<float*>(smem);       // the CTAs' partial sums [CTA][rank][row]
  float* s_warp = s_cta + kMaxCluster * F::kSums;      // the warps' [warp][rank][row]; later, to turn
  float (*s_turn)[kRows][F::kCols + 4] = reinterpret_cast<float (*)[kRows][F::kCols + 4]>(s_warp);
  // the intermediate's two parts
  __nv_bfloat16 (*s_u)[kRows][F::kPitch] =
      reinterpret_cast<__nv_bfloat16 (*)[kRows][F::kPitch]>(smem + F::kOffU);
  __shared__ int s_tmp[8 + kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int C = a.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  wait_for_launch_before();
  RowTile t;
  if (!find_tile<kThreads, kRows>(a.off, a.E, a.M, static_cast<int>(blockIdx.x) / C, s_tmp, a.status, t)) return;
  if (t.nrows == 0) return;
  const int K = a.K, N = a.N, R = a.R;
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.base);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  const int groups = (N + F::kCols - 1) / F::kCols;
  const int n0 = static_cast<int>(static_cast<long long>(groups) * rank / C);
  const int n1 = static_cast<int>(static_cast<long long>(groups) * (rank + 1) / C);
  // The output's rows that this lane stores: eight columns of row `lane / chunks + k * 32 / chunks`.
  constexpr int kChunks = F::kCols / 8, kSteps = kRows * kChunks / 32;
  int place[kSteps];
  int* status = rank == 0 && warp == 0 && lane % kChunks == 0 ? a.status : nullptr;
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int r = (lane + 32 * k) / kChunks;
    place[k] = r < t.nrows ? row_place(a.out_index, t.row0 + r, a.out_rows, status) : -1;
  }
  auto base_piece = [&](int group, int k) {
    const int c = group * F::kCols + lane % kChunks * 8;
    const bool there = base != nullptr && place[k] >= 0 && c < N;
    return there ? *reinterpret_cast<const uint4*>(base + static_cast<size_t>(place[k]) * N + c)
                 : make_uint4(0u, 0u, 0u, 0u);
  };

  if (t.e == a.E) {
    // Rows without an adapter: their base, or zeros.
    if (a.u != nullptr && rank == 0)
      for (int i = tid; i < t.nrows * R; i += kThreads) a.u[static_cast<size_t>(t.row0) * R + i] = 0.0f;
    if (out == base) return;
    for (int group = n0 + warp; group < n1; group += kWarps)
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int c = group * F::kCols + lane % kChunks * 8;
        const uint4 v = base_piece(group, k);
        if (place[k] >= 0 && c < N) *reinterpret_cast<uint4*>(out + static_cast<size_t>(place[k]) * N + c) = v;
      }
    return;
  }

  // ---------------------------------------------------- this CTA's columns of x and A
  // Lane (g, q): ranks g and g + 8 of a 16-rank tile, row g of x, columns 8 q .. of a 32-column block.
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(a.w1) + static_cast<size_t>(t.e) * R * K;
  const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(a.w2) + static_cast<size_t>(t.e) * N * R;
  const int xrow = g < t.nrows ? row_place(a.in_index, t.row0 + g, a.in_rows,
                                           rank == 0 && warp == 0 && q == 0 ? a.status : nullptr)
                               : -1;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.in) + static_cast<size_t>(xrow < 0 ? 0 : xrow) * K;
  const int kblocks = (K + 31) / 32;
  const int b0 = static_cast<int>(static_cast<long long>(kblocks) * rank / C);
  const int b1 = static_cast<int>(static_cast<long long>(kblocks) * (rank + 1) / C);
  float sum[2 * NB][4];
#pragma unroll
  for (int m = 0; m < 2 * NB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[m][i] = 0.0f;
  constexpr int kAhead = NB == 4 ? 1 : 2;
  for (int b = b0 + warp; b < b1; b += kAhead * kWarps) {
    uint4 xv[kAhead], top[kAhead][2 * NB], bottom[kAhead][2 * NB];
#pragma unroll
    for (int h = 0; h < kAhead; ++h) {
      const int col = 32 * (b + h * kWarps) + 8 * q;
      const bool there = b + h * kWarps < b1 && col < K;
      xv[h] = load16(x + col, there && xrow >= 0);
#pragma unroll
      for (int m = 0; m < 2 * NB; ++m) {
        const int j = 16 * m + g;
        top[h][m] = load16(A + static_cast<size_t>(j) * K + col, there && j < R);
        bottom[h][m] = load16(A + static_cast<size_t>(j + 8) * K + col, there && j + 8 < R);
      }
    }
#pragma unroll
    for (int h = 0; h < kAhead; ++h)
#pragma unroll
      for (int m = 0; m < 2 * NB; ++m) mma_32(sum[m], top[h][m], bottom[h][m], xv[h]);
  }
  // The first pieces of B and of base are on their way while the sums are exchanged.  (All of B's part
  // brought into L2 meanwhile, by bulk prefetch, cost 128 rows of 32 adapters of rank 64 17.2 -> 19.6 us.)  Lane (g, q):
  // columns g and g + 8 of a 16-column tile, ranks 8 q .. of a block.
  uint4 top[F::kTiles][NB], bottom[F::kTiles][NB], bv[kSteps];
  auto load_group = [&](int group) {
#pragma unroll
    for (int m = 0; m < F::kTiles; ++m) {
      const int n = group * F::kCols + 16 * m + g;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int j = 32 * b + 8 * q;
        top[m][b] = load16(B + static_cast<size_t>(n) * R + j, n < N && j < R);
        bottom[m][b] = load16(B + static_cast<size_t>(n + 8) * R + j, n + 8 < N && j < R);
      }
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) bv[k] = base_piece(group, k);
  };
  int group = n0 + warp;
  if (group < n1) load_group(group);
#pragma unroll
  for (int m = 0; m < 2 * NB; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      s_warp[warp * F::kSums + (16 * m + g + 8 * (i >> 1)) * kRows + 2 * q + (i & 1)] = sum[m][i];
  __syncthreads();
  if (C > 1) cluster_sync();  // every CTA of the cluster runs: its shared memory may be written
  for (int i = tid; i < F::kSums; i += kThreads) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_warp[w * F::kSums + i];
    const uint32_t at = smem_u32(&s_cta[rank * F::kSums + i]);
    for (int p = 0; p < C; ++p) st_cluster_f1(map_to_cta(at, p), v);
  }
  cluster_sync();
  const float scale = a.scale != nullptr ? a.scale[t.e] : 1.0f;
  for (int i = tid; i < F::kSums; i += kThreads) {
    const int j = i / kRows, r = i % kRows;
    float v = 0.0f;
    for (int p = 0; p < C; ++p) v += s_cta[p * F::kSums + i];
    const bool live = j < R && r < t.nrows;
    if (a.u != nullptr && rank == 0 && live) a.u[static_cast<size_t>(t.row0 + r) * R + j] = v;
    uint32_t hi, lo;
    split2(live ? v * scale : 0.0f, 0.0f, hi, lo);
    s_u[0][r][j] = __ushort_as_bfloat16(static_cast<unsigned short>(hi));
    s_u[1][r][j] = __ushort_as_bfloat16(static_cast<unsigned short>(lo));
  }
  __syncthreads();
  // ---------------------------------------------------- this CTA's columns of out
  uint4 u[2][NB];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int b = 0; b < NB; ++b) u[p][b] = *reinterpret_cast<const uint4*>(&s_u[p][g][32 * b + 8 * q]);
  for (; group < n1; group += kWarps) {
    float c[F::kTiles][4];
#pragma unroll
    for (int m = 0; m < F::kTiles; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i) c[m][i] = 0.0f;
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int b = 0; b < NB; ++b) mma_32(c[m], top[m][b], bottom[m][b], u[p][b]);
    }
    uint4 old[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) old[k] = bv[k];
    if (group + kWarps < n1) load_group(group + kWarps);
    __syncwarp();  // the group before has left the turning tile
#pragma unroll
    for (int m = 0; m < F::kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) s_turn[warp][2 * q + (i & 1)][16 * m + g + 8 * (i >> 1)] = c[m][i];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int r = (lane + 32 * k) / kChunks, at = lane % kChunks * 8;
      const int col = group * F::kCols + at;
      const float4* f = reinterpret_cast<const float4*>(&s_turn[warp][r][at]);
      const float4 y = f[0], z = f[1];
      const float2 o0 = unpack_bf16(old[k].x), o1 = unpack_bf16(old[k].y), o2 = unpack_bf16(old[k].z),
                   o3 = unpack_bf16(old[k].w);
      const uint4 v = make_uint4(pack_bf16(o0.x + y.x, o0.y + y.y), pack_bf16(o1.x + y.z, o1.y + y.w),
                                 pack_bf16(o2.x + z.x, o2.y + z.y), pack_bf16(o3.x + z.z, o3.y + z.w));
      if (place[k] >= 0 && col < N) *reinterpret_cast<uint4*>(out + static_cast<size_t>(place[k]) * N + col) = v;
    }
  }
}

cudaLaunchConfig_t config(int cluster, long long tiles, size_t smem, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.dynamicSmemBytes = smem;
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cluster));
  cfg.blockDim = dim3(kThreads);
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
template <int NB>
long long clusters_at_once(int c) {
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int active[kMaxCluster + 1];
  if (asked_ctx == 0 || asked_ctx != current_context_id()) {
    for (int k = 2; k <= kMaxCluster; ++k) {
      cudaLaunchAttribute attr[2] = {};
      const cudaLaunchConfig_t cfg = config(k, 1, Few<NB>::kSmem, attr);
      if (cudaOccupancyMaxActiveClusters(&active[k], lora_few_kernel<NB>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();  // a size that does not fit is no error of the call
        active[k] = 0;
      }
    }
    asked_ctx = current_context_id();
  }
  return active[c];
}

template <int NB>
cudaError_t launch(LoraArgs a, cudaStream_t stream) {
  static thread_local uint64_t attr_ctx = 0;
  const cudaError_t err =
      set_smem_attr_once(reinterpret_cast<const void*>(lora_few_kernel<NB>), Few<NB>::kSmem, &attr_ctx);
  if (err != cudaSuccess) return err;
  // At most this many tiles, one more for rows without an adapter included; about half a tile of each
  // adapter's is empty.
  const long long some = a.M < a.E ? a.M : a.E, full = (a.M + kRows - 1) / kRows;
  const long long tiles = full + some + 1, likely = full + some / 2;
  // As many CTAs to a tile as run at once.  Rank 16 of 64 adapters, 4096 x 4096, with one, two, four and
  // eight: 16 rows 13.2, 8.8, 6.9 and 6.0 us, 256 rows 16, 11, 9.2 and 13.4.
  const int most = a.max_cluster > 0 && a.max_cluster < kMaxCluster ? a.max_cluster : kMaxCluster;
  int c = 1;
  for (int k = 2; k <= most; k *= 2)
    if (likely <= clusters_at_once<NB>(k)) c = k;
  a.cluster = c;
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t cfg = config(c, tiles, Few<NB>::kSmem, attr);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, lora_few_kernel<NB>, a);
}

}  // namespace

// Here and in lora.cu, 4096 x 4096: eight adapters of rank 16, 1024 rows 13.1 and 14.2 us, 2048 rows 25 and 18;
// rank 64, 512 rows 14.4 and 14.6, 1024 rows 22 and 17.5; rank 128, 512 rows 21 and 17.6, 1024 rows 35 and 22.5,
// but of 64 adapters 512 rows 34 and 43, and 2048 x 1536 12.5 and 12.7.
bool lora_is_few(int M, int R) { return M <= (R <= 32 ? 1024 : 512); }

cudaError_t launch_lora_few(const LoraArgs& a, cudaStream_t stream) {
  if (a.R > 64) return launch<4>(a, stream);
  return a.R > 32 ? launch<2>(a, stream) : launch<1>(a, stream);
}

}  // namespace mgw
