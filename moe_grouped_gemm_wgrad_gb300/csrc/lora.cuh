// Device helpers of the low-rank adapter kernels (lora.cu, lora_grad.cu): bf16 tcgen05 products,
// operand tiles in either major order, gathered rows, and where a row tile lies.
//
// Every operand tile is a stack of 64-element, 128-byte rows in the 128-byte swizzle (8-row atoms
// of 1024 bytes), as a TMA box 64 elements wide writes them.  The tensor core reads such a tile
// either along its rows (K-major: the contraction runs within a row) or across them (MN-major: a
// row holds 64 neighbours of the product's M or N axis, the contraction runs from row to row).  So
// A [R, K] and B [N, R] serve both directions as they are stored, and one tile of x rows can be
// contracted over its features or over its tokens.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

#include "kernels.h"
#include "ptx.cuh"

namespace mgw {
namespace lora {

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int c0, int c1, int c2,
                                            uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
// 16 bytes global -> shared, asynchronously; zeros where `there` is false (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16u : 0u)
               : "memory");
}
// The calling thread's arrival on `bar`, by itself, once all its copies so far have landed.
__device__ __forceinline__ void copy_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// All of this thread's groups but the last `left` have landed.
__device__ __forceinline__ void copy_wait_left(int left) {
  switch (left) {
    case 0: copy_wait<0>(); break;
    case 1: copy_wait<1>(); break;
    case 2: copy_wait<2>(); break;
    case 3: copy_wait<3>(); break;
    case 4: copy_wait<4>(); break;
    case 5: copy_wait<5>(); break;
    case 6: copy_wait<6>(); break;
    case 7: copy_wait<7>(); break;
    case 8: copy_wait<8>(); break;
    case 9: copy_wait<9>(); break;
    default: copy_wait<10>(); break;
  }
}
// Waits, all lanes of a warp together, and says to all whether the phase came.
__device__ __forceinline__ bool wait_all(uint32_t bar, uint32_t parity, volatile int* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
}
__device__ __forceinline__ void give_up(volatile int* abort, int* status) {
  *abort = 1;
  if (status != nullptr) atomicOr(status, kDevTimeout);
}
// Orders generic-proxy accesses of any memory before later async-proxy ones (TMA, tcgen05).
__device__ __forceinline__ void fence_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// D[tmem] (+)= A[smem] B[smem]^T, bf16 operands, fp32 accumulators, K = 16.
__device__ __forceinline__ void mma_bf16(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f16: fp32 accumulate, bf16 x bf16, shape 128 x N; a set bit says
// that the operand is MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (8u << 24);
}
// A step of 16 along the contraction, in the descriptor's 16-byte units: 32 bytes within the rows
// of a K-major tile, 16 rows of an MN-major one.
constexpr uint32_t kStepK = 2, kStepMn = 128;
// MN-major tile: `block` bytes between its 64-wide column blocks (the leading offset), 1024 bytes
// between its 8-row groups.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t block) {
  return make_sdesc(saddr, block, 1024, 2);
}

// The launch before in the stream has ended and its results are there.  Kernels of this family are launched
// as programmatic dependents, the first of a call too, and wait before they touch memory that others
// write: launched one after the other they take their own time and 0.6 us each, where plain launches of a
// few us start at multiples of 2.05 us (6 us: 6.6 against 8.2).  Every thread waits before it ends, so
// that a launch that has ended has none before it still running.
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
inline cudaLaunchAttribute dependent_launch() {
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  return attr;
}

// cluster_sync in two halves; each by all threads of a warp together.
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_u4(uint32_t addr, uint4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_shared_f4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b), "f"(c), "f"(d)
               : "memory");
}
__device__ __forceinline__ void st_shared_u4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_u4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}
// 32 lanes x 16 columns of the warp's lane quarter.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
// Behind a tmem_wait_ld: keeps the uses of loaded registers there.
template <int N>
__device__ __forceinline__ void tmem_loaded(uint32_t (&r)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}
__device__ __forceinline__ bool mbar_wait_drain(uint32_t bar, uint32_t parity) {
  int never = 0;
  return mbar_wait(bar, parity, &never);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}
// v = hi + lo to 2^-17 of v: two bf16 parts, whose products with a bf16 operand are summed in the
// same fp32 accumulator, so that the rank-R intermediate loses nothing that a bf16 output shows.  An
// infinite v is all in hi (inf - inf would be none); lo is then 0.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  const float2 h = unpack_bf16(hi);
  const float la = fabsf(h.x) < INFINITY ? a - h.x : 0.0f;
  const float lb = fabsf(h.y) < INFINITY ? b - h.y : 0.0f;
  lo = pack_bf16(la, lb);
}

// Byte offset of 16-byte chunk c (0 .. 7) of row r in a tile of 128-byte swizzled rows.
__device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t c) { return r * 128u + ((c ^ (r & 7u)) << 4); }

struct RowTile {
  int e;      // adapter, or E for rows without one
  int row0;   // first row
  int nrows;  // 0: the tile does not exist
};

// The index-th tile of `kTile` rows, counting every adapter's tiles in turn and then those of the
// rows behind off[E].  Called by all threads of a block of kThreads; s_tmp holds 8 + kThreads / 32
// ints.  False (block-uniform, and the same in every block) where the offsets are not
// 0 = off[0] <= .. <= off[E] <= M: that is reported once per block.
template <int kThreads, int kTile>
__device__ __forceinline__ bool find_tile(const int32_t* __restrict__ off, int E, int M, int index, int* s_tmp,
                                          int* status, RowTile& t) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (E + kThreads - 1) / kThreads;
  const int e0 = min(tid * per, E), e1 = min(e0 + per, E);
  int tiles = 0, bad = 0;
  int lo = off[e0];
  if (tid == 0) {
    s_tmp[0] = E, s_tmp[1] = 0, s_tmp[2] = 0;
    bad = lo != 0;
    bad |= off[E] > M;
  }
  const int first = lo;
  for (int e = e0; e < e1; ++e) {
    const int hi = off[e + 1];
    bad |= hi < lo;
    tiles += (hi - lo + kTile - 1) / kTile;
    lo = hi;
  }
  if (__syncthreads_or(bad)) {
    if (tid == 0 && status != nullptr) atomicOr(status, kDevBadOffsets);
    return false;
  }
  int before = tiles;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += y;
  }
  if (lane == 31) s_tmp[8 + warp] = before;
  before -= tiles;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    const int n = s_tmp[8 + w];
    if (w < warp) before += n;
    total += n;
  }
  if (index >= before && index < before + tiles) {
    int at = before, start = first;
    for (int e = e0; e < e1; ++e) {
      const int end = off[e + 1];
      const int n = (end - start + kTile - 1) / kTile;
      if (index < at + n) {
        const int r = (index - at) * kTile;
        s_tmp[0] = e;
        s_tmp[1] = start + r;
        s_tmp[2] = min(kTile, end - start - r);
        break;
      }
      at += n;
      start = end;
    }
  }
  if (tid == 0 && index >= total) {
    const long long r = static_cast<long long>(off[E]) + static_cast<long long>(index - total) * kTile;
    if (r < M) {
      s_tmp[1] = static_cast<int>(r);
      s_tmp[2] = min(kTile, M - static_cast<int>(r));
    }
  }
  __syncthreads();
  t.e = s_tmp[0];
  t.row0 = s_tmp[1];
  t.nrows = s_tmp[2];
  return true;
}

// Row r's place: itself, or index[r]; -1 where that lies outside [0, rows) (reported).
__device__ __forceinline__ int row_place(const int32_t* __restrict__ index, int r, int rows, int* status) {
  int i = r;
  if (index != nullptr) {
    i = index[r];
    if (i < 0 || i >= rows) {
      if (status != nullptr) atomicOr(status, kDevBadIndex);
      i = -1;
    }
  }
  return i;
}

}  // namespace lora
}  // namespace mgw
