// Backward pass of the expert product's epilogue:
//
//   dz[r, n]    = dy[r, n] act'(z[r, n])     (gated: d gate = dy up act'(gate), d up = dy act(gate))
//   dbias[e, n] = sum over the rows r of expert e of dz[r, n]
//
// One CTA per (128-row tile of one expert, 256 columns): 8 warps take the tile's rows in turn,
// a lane 8 columns (16-byte loads and stores), and keep the columns' sums in fp32 registers.
// With dbias the warps' sums meet in shared memory and go to the workspace, one row of sums
// per tile; a second launch adds every expert's tiles in order, so dbias does not vary between
// runs.  dbias sums dz before it is rounded to bf16.  HBM bounds it: z, dy and dz once each.
#include <cuda_bf16.h>

#include <cstdint>

#include "act.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mgw {
namespace {

constexpr int kRows = 128;   // rows of a tile
constexpr int kCols = 256;   // columns per CTA: 32 lanes x 8
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
template <int ACT>
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
  if (tile >= s_pad[a.E] / kRows) return;
  const int e = locate(tile * kRows, s_pad, a.E);
  const int first = tile * kRows - s_pad[e];
  const int rows = min(kRows, s_off[e + 1] - s_off[e] - first);
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
    for (int r = warp; r < rows; r += kWarps) {
      const long long row = row0 + r;
      float g[8], zv[8], d[8];
      unpack8(*reinterpret_cast<const uint4*>(dy + row * F + c), g);
      if constexpr (kGated) {
        float up[8], du[8];
        unpack8(*reinterpret_cast<const uint4*>(z + row * a.N + c), zv);
        unpack8(*reinterpret_cast<const uint4*>(z + row * a.N + F + c), up);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float v, sl;
          act_value_slope<kInner>(zv[i], v, sl);
          d[i] = g[i] * up[i] * sl;
          du[i] = g[i] * v;
          sum[0][i] += d[i];
          sum[kSums - 1][i] += du[i];
        }
        *reinterpret_cast<uint4*>(dz + row * a.N + c) = pack8(d);
        *reinterpret_cast<uint4*>(dz + row * a.N + F + c) = pack8(du);
      } else {
        if constexpr (ACT != kActNone) {
          unpack8(*reinterpret_cast<const uint4*>(z + row * a.N + c), zv);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float v, sl;
            act_value_slope<kInner>(zv[i], v, sl);
            d[i] = g[i] * sl;
          }
          *reinterpret_cast<uint4*>(dz + row * a.N + c) = pack8(d);
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = g[i];
          if (dz != nullptr) *reinterpret_cast<uint4*>(dz + row * a.N + c) = pack8(d);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[0][i] += d[i];
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
      a.partial[static_cast<size_t>(tile) * a.N + s * F + col] = v;
    }
  }
}

// dbias[e, n]: the sums of the expert's tiles, in tile order.
__global__ void __launch_bounds__(256) act_dbias_kernel(ActBwdArgs a) {
  extern __shared__ int s_tab[];
  __shared__ int s_flag;
  int* s_off = s_tab;
  int* s_pad = s_tab + a.E + 1;
  if (!load_offsets(a.expert_off, a.E, a.M, s_off, s_pad, &s_flag, nullptr)) return;
  const int e = blockIdx.x;
  const int n = blockIdx.y * blockDim.x + threadIdx.x;
  if (n >= a.N) return;
  float v = 0.0f;
  for (int t = s_pad[e] / kRows; t < s_pad[e + 1] / kRows; ++t)
    v += a.partial[static_cast<size_t>(t) * a.N + n];
  a.dbias[static_cast<size_t>(e) * a.N + n] = v;
}

template <int ACT>
cudaError_t launch(const ActBwdArgs& a, cudaStream_t stream) {
  const int F = act_gated(ACT) ? a.N / 2 : a.N;
  const size_t smem = sizeof(int) * 2 * (static_cast<size_t>(a.E) + 1);
  const long long experts = a.M < a.E ? a.M : a.E;
  const long long tiles = a.M / kRows + experts;
  const dim3 grid(static_cast<unsigned>(tiles > 0 ? tiles : 1), static_cast<unsigned>((F + kCols - 1) / kCols));
  act_backward_kernel<ACT><<<grid, kWarps * 32, smem, stream>>>(a);
  const cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess || a.dbias == nullptr) return err;
  const dim3 grid2(static_cast<unsigned>(a.E), static_cast<unsigned>((a.N + 255) / 256));
  act_dbias_kernel<<<grid2, 256, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

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
