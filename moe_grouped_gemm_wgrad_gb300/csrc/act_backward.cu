// Backward pass of the expert product's epilogue:
//
//   dz[r, n]    = dy[r, n] act'(z[r, n])     (gated: d gate = dy up act'(gate), d up = dy act(gate))
//   dbias[e, n] = sum over the rows r of expert e of dz[r, n]
//
// One CTA per (128-row tile of one expert, 256 columns): 8 warps take the tile's rows in turn,
// a lane 8 columns (16-byte loads and stores), and keep the columns' sums in fp32 registers.  A
// warp asks for four rows before it works on the first: 65536 x 1536 took 115 us with one row at
// a time, 104 us so (tiles of 64 or 32 rows: no gain at any size).
//
// With dbias the warps' sums meet in shared memory and go to the workspace, one row of sums per
// tile; a second launch adds every expert's tiles in an order that the sizes fix, so dbias does
// not vary between runs.  It sums dz before dz is rounded to bf16.  Up to kWholeRows rows in all,
// a CTA takes a whole expert instead and stores its dbias itself: one launch and no workspace (a
// launch costs more than the few rows do).
//
// HBM bounds it: z, dy and dz once each.  65536 x 1536 GELU: 94 us without dbias (6.4 TB/s, 96%
// of the copy rate), 100 us with it.
#include <cuda_bf16.h>

#include <cstdint>

#include "act.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mgw {
namespace {

constexpr int kRows = 128;   // rows of a tile
constexpr int kCols = 256;   // columns per CTA: 32 lanes x 8
constexpr int kWholeRows = 512;
constexpr int kWarps = 8;

__device__ __forceinline__ void unpack8(uint4 u, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(h[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint4 u;
  __nv_bfloat162* h = reinterpret_cast<__nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  return u;
}

// The largest e with first[e] <= i.
__device__ __forceinline__ int locate(int i, const int* first, int E) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= i)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// Columns are those of dy: F = N, or N / 2 when gated (then each lane has a gate and an up
// column).  Tiles are counted on the 128-padded row axis.
// WHOLE: blockIdx.x is an expert, not a row tile.
template <int ACT, bool WHOLE>
__global__ void __launch_bounds__(kWarps * 32) act_backward_kernel(ActBwdArgs a) {
  constexpr bool kGated = act_gated(ACT);
  constexpr int kInner = act_inner(ACT);
  constexpr int kSums = kGated ? 2 : 1;
  extern __shared__ int s_tab[];
  __shared__ int s_flag;
  __shared__ float s_sum[kWarps][kCols];
  int* s_off = s_tab;
  int* s_pad = s_tab + a.E + 1;
  if (!load_offsets(a.expert_off, a.E, a.M, s_off, s_pad, &s_flag, a.status)) return;
  const int tile = blockIdx.x;
  int e, first = 0, rows;
  if constexpr (WHOLE) {
    e = tile;
    rows = s_off[e + 1] - s_off[e];
  } else {
    if (tile >= s_pad[a.E] / kRows) return;
    e = locate(tile * kRows, s_pad, a.E);
    first = tile * kRows - s_pad[e];
    rows = min(kRows, s_off[e + 1] - s_off[e] - first);
  }
  const long long row0 = s_off[e] + first;
  const int warp = threadIdx.x >> 5;
  const int F = kGated ? a.N / 2 : a.N;
  const int c = blockIdx.y * kCols + static_cast<int>(lane_id()) * 8;
  const __nv_bfloat16* dy = static_cast<const __nv_bfloat16*>(a.dy);
  const __nv_bfloat16* z = static_cast<const __nv_bfloat16*>(a.z);
  __nv_bfloat16* dz = static_cast<__nv_bfloat16*>(a.dz);
  float sum[kSums][8];
#pragma unroll
  for (int s = 0; s < kSums; ++s)
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[s][i] = 0.0f;
  if (c < F) {
    constexpr int kAhead = 4;
    for (int r0 = warp; r0 < rows; r0 += kWarps * kAhead) {
      uint4 gr[kAhead], zr[kAhead], ur[kGated ? kAhead : 1];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        // past the tile's last row: its own first one again, which is not stored or summed
        const long long row = row0 + (r0 + kWarps * i < rows ? r0 + kWarps * i : r0);
        gr[i] = *reinterpret_cast<const uint4*>(dy + row * F + c);
        if constexpr (ACT != kActNone) zr[i] = *reinterpret_cast<const uint4*>(z + row * a.N + c);
        if constexpr (kGated) ur[i] = *reinterpret_cast<const uint4*>(z + row * a.N + F + c);
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (r0 + kWarps * i >= rows) break;
        const long long row = row0 + r0 + kWarps * i;
        float g[8], d[8];
        unpack8(gr[i], g);
        if constexpr (ACT == kActNone) {
#pragma unroll
          for (int j = 0; j < 8; ++j) d[j] = g[j];
          if (dz != nullptr) *reinterpret_cast<uint4*>(dz + row * a.N + c) = pack8(d);
        } else {
          float zv[8];
          unpack8(zr[i], zv);
          float up[8], du[8];
          if constexpr (kGated) unpack8(ur[i], up);
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            float v[2], sl[2];
            act_value_slope2<kInner>(zv[j], zv[j + 1], v, sl);
#pragma unroll
            for (int i2 = 0; i2 < 2; ++i2) {
              d[j + i2] = g[j + i2] * sl[i2];
              if constexpr (kGated) {
                d[j + i2] *= up[j + i2];
                du[j + i2] = g[j + i2] * v[i2];
                sum[kSums - 1][j + i2] += du[j + i2];
              }
            }
          }
          *reinterpret_cast<uint4*>(dz + row * a.N + c) = pack8(d);
          if constexpr (kGated) *reinterpret_cast<uint4*>(dz + row * a.N + F + c) = pack8(du);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[0][j] += d[j];
      }
    }
  }
  if (a.dbias == nullptr) return;
#pragma unroll
  for (int s = 0; s < kSums; ++s) {
    if (s > 0) __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) s_sum[warp][lane_id() * 8 + i] = sum[s][i];
    __syncthreads();
    const int col = blockIdx.y * kCols + threadIdx.x;
    if (col < F) {
      float v = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += s_sum[w][threadIdx.x];
      (WHOLE ? a.dbias + static_cast<size_t>(e) * a.N : a.partial + static_cast<size_t>(tile) * a.N)[s * F + col] = v;
    }
  }
}

// dbias[e, n]: the sums of the expert's tiles.  The CTA's 8 warps are 8 / SLICES column blocks
// of 32 by SLICES slices of the tiles (tiles s, s + SLICES, ..), whose sums are added in order.
template <int SLICES>
__global__ void __launch_bounds__(kWarps * 32) act_dbias_kernel(ActBwdArgs a) {
  constexpr int kBlocks = kWarps / SLICES;
  __shared__ int s_first;
  __shared__ float s_sum[kWarps][32];
  const int e = blockIdx.x, warp = threadIdx.x >> 5;
  const int slice = warp / kBlocks;
  const int n = (blockIdx.y * kBlocks + warp % kBlocks) * 32 + static_cast<int>(lane_id());
  if (threadIdx.x == 0) s_first = 0;
  __syncthreads();
  // the expert's first tile on the padded axis, and the offsets' check, in one pass
  int bad = threadIdx.x == 0 && (a.expert_off[0] != 0 || a.expert_off[a.E] != a.M), before = 0;
  for (int i = threadIdx.x; i < a.E; i += blockDim.x) {
    const int c = a.expert_off[i + 1] - a.expert_off[i];
    bad |= c < 0;
    if (i < e) before += (c + 127) & ~127;
  }
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane_id() == 0 && before != 0) atomicAdd(&s_first, before);
  if (__syncthreads_or(bad)) return;
  const int t0 = s_first / kRows;
  const int t1 = t0 + (a.expert_off[e + 1] - a.expert_off[e] + kRows - 1) / kRows;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the partial sums are there
  float v = 0.0f;
  if (n < a.N) {
#pragma unroll 8
    for (int t = t0 + slice; t < t1; t += SLICES) v += a.partial[static_cast<size_t>(t) * a.N + n];
  }
  if constexpr (SLICES > 1) {
    s_sum[warp][lane_id()] = v;
    __syncthreads();
    if (slice != 0) return;
#pragma unroll
    for (int k = 1; k < SLICES; ++k) v += s_sum[warp + k * kBlocks][lane_id()];
  }
  if (n < a.N) a.dbias[static_cast<size_t>(e) * a.N + n] = v;
}

template <int SLICES>
cudaError_t launch_dbias(const ActBwdArgs& a, cudaStream_t stream) {
  constexpr int kBlockCols = kWarps / SLICES * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.E), static_cast<unsigned>((a.N + kBlockCols - 1) / kBlockCols));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = stream;
  // starts its own checks while the tiles' launch ends (programmatic dependent launch)
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, act_dbias_kernel<SLICES>, a);
}

template <int ACT>
cudaError_t launch(const ActBwdArgs& a, cudaStream_t stream) {
  const int F = act_gated(ACT) ? a.N / 2 : a.N;
  const size_t smem = sizeof(int) * 2 * (static_cast<size_t>(a.E) + 1);
  if (a.M <= kWholeRows && a.dbias != nullptr) {
    const dim3 grid(static_cast<unsigned>(a.E), static_cast<unsigned>((F + kCols - 1) / kCols));
    act_backward_kernel<ACT, true><<<grid, kWarps * 32, smem, stream>>>(a);
    return cudaGetLastError();
  }
  const long long experts = a.M < a.E ? a.M : a.E;
  const long long tiles = a.M / kRows + experts;
  const dim3 grid(static_cast<unsigned>(tiles > 0 ? tiles : 1), static_cast<unsigned>((F + kCols - 1) / kCols));
  act_backward_kernel<ACT, false><<<grid, kWarps * 32, smem, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || a.dbias == nullptr) return err;
  // Slices by the tiles an expert has on average: many CTAs cost more than a few loads in a row
  // (32768 x 1536 over 64 experts, profiled: 8.3 us with eight slices, 7.6 with one).  The host does
  // not know the largest expert: one far above the mean has its tiles added by fewer warps than
  // would be best.  65536 x 1536 GELU over 64 experts, events around a call: 110 us balanced, 124
  // with a third of the rows in one expert, 130 with half, 113 with all.
  const long long mean = tiles / a.E;
  if (mean >= 64) return launch_dbias<8>(a, stream);
  if (mean >= 16) return launch_dbias<2>(a, stream);
  return launch_dbias<1>(a, stream);
}

}  // namespace

size_t act_backward_workspace_bytes(int E, int M, int N) {
  if (M <= kWholeRows) return 0;
  // one row of sums per 128-row tile of an expert
  const size_t tiles = static_cast<size_t>(M) / kRows + static_cast<size_t>(M < E ? M : E);
  return sizeof(float) * tiles * static_cast<size_t>(N);
}

cudaError_t launch_act_backward(const ActBwdArgs& a, int act, cudaStream_t stream) {
  switch (act) {
    case kActNone: return launch<kActNone>(a, stream);
    case kActRelu: return launch<kActRelu>(a, stream);
    case kActGelu: return launch<kActGelu>(a, stream);
    case kActSilu: return launch<kActSilu>(a, stream);
    case kActSwiglu: return launch<kActSwiglu>(a, stream);
    case kActGeglu: return launch<kActGeglu>(a, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mgw
