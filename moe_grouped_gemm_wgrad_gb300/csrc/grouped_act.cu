// Grouped MXFP8 product with bias, activation and residual in its epilogue:
//
//   z[r, n] = sum_k x[r, k] W[e(r)][n, k] + bias[e(r), n]
//   y[r, :] = act(z[r, :]) + residual[r, :]          (gated: act(z[:, :F]) * z[:, F:])
//
// The weights are the tensor cores' M side and the routed rows the N side: D^T = W x^T.  An
// expert's rows then need no padding to a tile: they are cut into ceil(c / 208) tiles of equal
// width w (a multiple of 16), and the MMA's N is w.  A 1024-row expert runs as 5 tiles of 208
// instead of 8 of 128, and a decode step's few rows cost an N of 16, so its time is that of
// reading the weights.  In the accumulator a TMEM lane is an output feature and a column is a
// row of x; the epilogue turns 16-column groups by stmatrix.trans into row-major 16-byte
// pieces, so rows past the expert's last one are masked per piece.
//
// A CTA pair (tcgen05 cta_group::2) owns 256 weight rows (128 per CTA) x w routed rows (w / 2
// of them staged per CTA).  Gated products take 128 gate and 128 up rows per pair, interleaved
// in blocks of 16 (TMA boxes of 16 rows): lanes 0-15 of a TMEM lane quarter are gate rows and
// lanes 16-31 the same features' up rows, so the two 16-lane loads of a group give every thread
// the gate and the up value of its elements.
//
// TMEM: two accumulators of 208 columns (the epilogue of one item overlaps the MMAs of the
// next; 2 x 256 columns would leave no room for scale factors) and six 16-column scale slots.
//
// Roles (576 threads per CTA):
//   warp 0       TMA producer (both CTAs): weight rows, half of the routed rows, scale atoms.
//   warp 1       MMA issuer (even CTA).
//   warps 2-13   epilogue: three warps per TMEM lane quarter, taking 16-column groups in turn.
//                A group is a chain of waits (TMEM, staging tile, stores), so the number of
//                warps counts: with two per quarter 32768 rows of SwiGLU with residual and saved
//                pre-activation took 152 us, with three 138, with four no less.
//   warps 14-17  scale writers, one TMEM lane quarter each: they place the stage's scale words
//                in TMEM, which is what lets a tile start at any multiple of 16 rows and the
//                gate / up rows interleave.
//
// Measured on a GB300, isolated launches: 65536 x 1536 x 4096 over 64 experts 261 us without an
// epilogue (3.16 PFLOP/s, tensor pipe 80-87% busy), 280 us with GELU and saved pre-activation;
// back to back the power cap (SM clock 1.3 GHz) makes that 306 and 330 us.  128 rows over 64
// experts of 2048 x 4096: 85 us, 6.0 TB/s of weights.  Contractions below about 1500 are bound
// by the epilogue (65536 x 1024 x 256 over 16 experts, GELU, pre-activation saved: 73 to 81 us
// from process to process, HBM floor 43).
#include <cuda_bf16.h>

#include <cstdint>

#include "act.cuh"
#include "common.cuh"
#include "kernels.h"

namespace mgw {
namespace {

constexpr int kW = 208;       // widest row tile (MMA N)
constexpr int BL = 128;       // contraction elements per pipeline stage
constexpr int kStages = 6;
constexpr int kABytes = 128 * BL;              // this CTA's 128 weight rows
constexpr int kBBytes = (kW / 2) * BL;         // this CTA's half of the routed rows
constexpr int kStageBytes = kABytes + kBBytes; // 29 KB, 1024-aligned
constexpr int kSfA = 1024;                     // weight scale atoms (two when gated)
constexpr int kSfB = 1536;                     // scale atoms covering 208 rows from any start
constexpr int kSfStage = kSfA + kSfB;
constexpr int kOffSf = kStages * kStageBytes;
constexpr int kOffBar = kOffSf + kStages * kSfStage;
// full[], empty[], sf_full[], acc_full[2], acc_empty[2], done
constexpr int kNumBars = 3 * kStages + 5;
constexpr int kOffMisc = (kOffBar + kNumBars * 8 + 15) & ~15;
constexpr int kEpiParts = 3;  // epilogue warps per TMEM lane quarter
constexpr int kEpiWarps = 4 * kEpiParts;
// Per epilogue warp: a staging tile of 16 rows by 32 features in bf16 (gated: two of 16).
constexpr int kTurnBytes = 16 * 64;
// Most rows of an item whose contraction is split over the pairs of a cluster, and most pairs.
constexpr int kSplitRows = 64;
constexpr int kMaxSplit = 4;
static_assert((kMaxSplit - 1) * (kSplitRows / 16) * 4 * 2048 <= kStages * kStageBytes, "partial accumulators");
constexpr int kOffTurn = kOffMisc + 16;
constexpr int kOffTable = kOffTurn + kEpiWarps * kTurnBytes;
constexpr int kSfWarp0 = 2 + kEpiWarps;
constexpr int kThreads = (kSfWarp0 + 4) * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kSfCol0 = 2 * kW;
static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
static_assert(kSfCol0 + 16 * kStages <= kTmemCols, "TMEM budget");

// Tables: expert_off, padded starts, first row tile and row tile width of every expert, E+1 ints
// each.
__host__ __device__ constexpr size_t act_smem_bytes(int E) {
  return static_cast<size_t>(kOffTable) + sizeof(int) * 4 * (static_cast<size_t>(E) + 1) + 1024;
}
static_assert(act_smem_bytes(kMaxExperts) <= 232448, "shared memory budget");

__device__ __forceinline__ void mbar_wait_drain(uint32_t bar, uint32_t parity) {
  int never = 0;
  (void)mbar_wait(bar, parity, &never);
}
__device__ __forceinline__ void tmem_st_x4(uint32_t taddr, const uint32_t (&v)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// 16 lanes x 16 columns: r[4 b + 2 h + i] is lane lane_id / 4 + 8 h, column 8 b + 2 (lane_id % 4) + i.
__device__ __forceinline__ void tmem_ld_16x256b_x2(uint32_t taddr, uint32_t* r) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
                 "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
// Waits for the loads into r; naming r keeps its uses behind the wait.
__device__ __forceinline__ void tmem_wait_ld_regs(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
// Four 8 x 8 matrices of 16-bit values between fragments (lane l: row l / 4, columns
// 2 (l % 4) + {0, 1}) and shared memory, transposed: lane l gives the address of memory row
// l % 8 of matrix l / 8.
__device__ __forceinline__ void stmatrix_x4_trans(uint32_t addr, const uint32_t* r) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr),
               "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3])
               : "memory");
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_bf16(uint32_t u) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u));
}

// A warp's staging tile of 16 rows x CH 16-byte chunks of features.  Row r's chunk c lies at chunk
// c ^ swizzle(r) of its row, so that the 8 rows of a matrix (one chunk each) and the 8 lanes of a
// 16-byte access (whole rows) both meet the 8 bank groups once.  (With padded rows instead, 80
// bytes apart, the loads conflicted and kept the LSU's data pipe 62% busy.)
template <int CH>
struct Turn {
  static constexpr uint32_t kRow = 16 * CH;  // bytes
  static __device__ __forceinline__ uint32_t at(uint32_t r, uint32_t c) {
    return r * kRow + ((c ^ (CH == 4 ? (r >> 1) & 3u : (r >> 2) & 1u)) << 4);
  }
  // The memory rows' addresses this lane gives for matrices (8 rows, chunk): rows 0-7 of chunks
  // 0 .. 3 and, 8 rows on, the same again (CH == 4); all four (rows, chunk) at once (CH == 2).
  static __device__ __forceinline__ uint32_t fragment() {
    const uint32_t l = lane_id();
    return CH == 4 ? at(l & 7u, l >> 3) : at((l & 7u) + 8u * (l >> 4), (l >> 3) & 1u);
  }
  // Fragment f[4 b + i] of rows 8 b .., chunk i (CH == 4), or f[2 b + i] (CH == 2).
  static __device__ __forceinline__ void put(uint32_t frag, const uint32_t* f) {
    stmatrix_x4_trans(frag, f);
    if constexpr (CH == 4) stmatrix_x4_trans(frag + 8 * kRow, f + 4);  // 8 rows on: same swizzle
  }
  static __device__ __forceinline__ void get(uint32_t frag, uint32_t* f) {
    ldmatrix_x4_trans(frag, f);
    if constexpr (CH == 4) ldmatrix_x4_trans(frag + 8 * kRow, f + 4);
  }
  // This lane's pieces: rows lane / CH (+ 8 with CH == 4), chunk lane % CH.
  static __device__ __forceinline__ int row() { return static_cast<int>(lane_id() / CH); }
  static __device__ __forceinline__ int col() { return static_cast<int>(lane_id() % CH) * 8; }
  static __device__ __forceinline__ uint32_t piece() { return at(lane_id() / CH, lane_id() % CH); }
  // m: this lane's piece of the group's first row; left: rows of the group that exist.
  static __device__ __forceinline__ void store(uint32_t piece, __nv_bfloat16* m, size_t pitch, int left) {
#pragma unroll
    for (int p = 0; p < CH / 2; ++p) {
      const uint4 v = ld_shared_v4(piece + p * 8 * kRow);
      if (row() + 8 * p < left) *reinterpret_cast<uint4*>(m + 8 * p * pitch) = v;
    }
  }
  static __device__ __forceinline__ void load(const __nv_bfloat16* m, size_t pitch, int left,
                                              uint4 (&v)[CH / 2]) {
#pragma unroll
    for (int p = 0; p < CH / 2; ++p) {
      v[p] = make_uint4(0u, 0u, 0u, 0u);
      if (row() + 8 * p < left) v[p] = *reinterpret_cast<const uint4*>(m + 8 * p * pitch);
    }
  }
  static __device__ __forceinline__ void fill(uint32_t piece, const uint4 (&v)[CH / 2]) {
#pragma unroll
    for (int p = 0; p < CH / 2; ++p) st_shared_v4(piece + p * 8 * kRow, v[p]);
  }
};

// One work item: an expert's row tile x 256 weight rows.
struct Item {
  int e;      // expert
  int ft;     // feature tile
  int row0;   // first routed row
  int p0;     // its row on the padded axis
  int nrows;  // rows of the tile (1 .. 208)
  int width;  // nrows rounded up to 16: the MMA's N
};

// Walks a pair's items (expert-major, then row tile, then feature tile; items first, first + step,
// ..).  Every warp of the CTA walks the same sequence, so a step is kept short: no division, and
// the expert is searched for from the last one on.
struct Items {
  const int *s_off, *s_pad, *s_tile, *s_width;
  int tiles_f, total;        // feature tiles; items in all
  int step_t, step_f, step;  // the step in row tiles and feature tiles
  int it, t, ft, e;

  __device__ __forceinline__ Items(const int* off, const int* pad, const int* tile, const int* width,
                                   int tiles_f_, int total_, int first, int step_)
      : s_off(off), s_pad(pad), s_tile(tile), s_width(width), tiles_f(tiles_f_), total(total_),
        step_t(step_ / tiles_f_), step_f(step_ % tiles_f_), step(step_), it(first),
        t(first / tiles_f_), ft(first % tiles_f_), e(0) {}

  // The next item with rows; false past the last one.  The values are the same in every lane.
  __device__ __forceinline__ bool next(Item& x) {
    while (it < total) {
      while (s_tile[e + 1] <= t) ++e;  // t < s_tile[E]
      e = __shfl_sync(0xffffffffu, e, 0);
      const int w = s_width[e];
      const int r = (t - s_tile[e]) * w;
      x.e = e;
      x.ft = ft;
      x.row0 = __shfl_sync(0xffffffffu, s_off[e] + r, 0);
      x.p0 = __shfl_sync(0xffffffffu, s_pad[e] + r, 0);
      // rounding w up can leave a last tile without rows
      x.nrows = __shfl_sync(0xffffffffu, max(min(w, s_off[e + 1] - s_off[e] - r), 0), 0);
      x.width = (x.nrows + 15) & ~15;
      it += step;
      t += step_t;
      ft += step_f;
      if (ft >= tiles_f) ft -= tiles_f, ++t;
      if (x.nrows > 0) return true;
    }
    return false;
  }
};

// S > 1: few items of few rows.  A cluster of S pairs takes one item, pair j the j-th part of the
// contraction; the other pairs' accumulators go to the first pair's ring, which is idle by then,
// and are added there in pair order.
template <int ACT, int S>
__global__ void __launch_bounds__(kThreads, 1) grouped_act_kernel(const __grid_constant__ ActMmArgs args) {
  constexpr bool kGated = act_gated(ACT);
  constexpr int kInner = act_inner(ACT);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int E = args.E;
  int* s_misc = reinterpret_cast<int*>(smem + kOffMisc);  // [0] tmem base [1] abort [2] flag
  int* s_off = reinterpret_cast<int*>(smem + kOffTable);
  int* s_pad = s_off + (E + 1);
  int* s_tile = s_pad + (E + 1);
  int* s_width = s_tile + (E + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(&s_misc[1]);
  const int tid = threadIdx.x;
  // The same value in every lane, in a form the compiler knows to be: the producer and the MMA
  // warp then keep addresses, descriptors and coordinates in uniform registers, which is what
  // their TMA and tcgen05 instructions take.
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t lane = lane_id();
  const uint32_t cta = cluster_ctarank();
  const uint32_t rank = cta & 1u;   // in the pair; 0 issues the pair MMAs
  const uint32_t even = cta & ~1u;  // the pair's even CTA
  const bool leader = rank == 0;

  if (tid == 0) s_misc[1] = 0;
  // Both CTAs read the same offsets, so both return here or neither does.
  if (!load_offsets(args.expert_off, E, args.M, s_off, s_pad, &s_misc[2], args.status)) return;

  const uint32_t bar0 = sbase + kOffBar;
  auto bar_full = [&](int st) { return bar0 + 8u * st; };                   // even CTA
  auto bar_empty = [&](int st) { return bar0 + 8u * (kStages + st); };
  auto bar_sf_full = [&](int st) { return bar0 + 8u * (2 * kStages + st); };
  auto bar_acc_full = [&](int b) { return bar0 + 8u * (3 * kStages + b); };
  auto bar_acc_empty = [&](int b) { return bar0 + 8u * (3 * kStages + 2 + b); };  // even CTA
  const uint32_t bar_done = bar0 + 8u * (3 * kStages + 4);
  if (warp == 0) {
    // first row tile of every expert: an exclusive scan of ceil(count / 208)
    int carry = 0;
    if (lane == 0) s_tile[0] = 0;
    for (int base = 0; base < E; base += 32) {
      const int e = base + static_cast<int>(lane);
      const int cnt = e < E ? s_off[e + 1] - s_off[e] : 0;
      int v = (cnt + kW - 1) / kW;
      if (e < E) s_width[e] = v > 0 ? ((cnt + v - 1) / v + 15) & ~15 : 16;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= static_cast<uint32_t>(d)) v += y;
      }
      if (e < E) s_tile[e + 1] = carry + v;
      carry += __shfl_sync(0xffffffffu, v, 31);
    }
  } else if (warp == 1) {
    tmem_alloc_pair(smem_u32(&s_misc[0]), kTmemCols);
    tmem_relinquish_pair();
  } else if (warp == 2 && lane == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(bar_full(st), 1 + 8);  // the operands' bytes, and four writer warps in each CTA
      mbar_init(bar_empty(st), 1);
      mbar_init(bar_sf_full(st), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar_acc_full(b), 1);
      mbar_init(bar_acc_empty(b), 2 * kEpiWarps);
    }
    mbar_init(bar_done, 1);
    fence_mbar_init();
    tma_prefetch_desc(&args.tm_w);
    tma_prefetch_desc(&args.tm_x);
    tma_prefetch_desc(&args.tm_x16);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are initialised before any remote arrive
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(__shfl_sync(0xffffffffu, s_misc[0], 0));
  auto abort_both = [&]() {
    *abort_flag = 1;
    for (uint32_t i = 0; i < 2 * S; ++i)
      if (i != cta) st_cluster_u32(map_to_cta(smem_u32(&s_misc[1]), i), 1u);
    if (args.status) atomicOr(args.status, kDevTimeout);
  };

  const int N = args.N;
  const int F = kGated ? N / 2 : N;  // output columns
  const int tiles_f = N / 256;
  const int nch = args.K / BL;
  const int total = __shfl_sync(0xffffffffu, s_tile[E], 0) * tiles_f;  // < 2^31: the C ABI checks the sizes
  // first item and step to the next one; with S > 1 a cluster has one item at most
  const int pair = static_cast<int>(blockIdx.x) / (2 * S);
  const int npairs = S > 1 ? 1 << 30 : static_cast<int>(gridDim.x >> 1);
  Items items(s_off, s_pad, s_tile, s_width, tiles_f, total, pair, npairs);
  // this pair's chunks of the contraction
  const int split = static_cast<int>(cta >> 1);
  const int c0 = nch * split / S, c1 = nch * (split + 1) / S;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // The whole warp walks the loop, one lane issues (measured against one lane walking it
    // alone: 38 instead of 103 cycles per copy, and 164 instead of 400 per four MMAs).
    const bool issue = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    uint32_t chunks = 0;
    bool ok = true;
    const uint32_t full0_leader = map_to_cta(bar_full(0), even);
    const long long a_tiles = args.Mw / 128;   // 128-row tiles of the weights' scale layout
    const long long b_tiles = args.Mcap / 128;
    Item x;
    while (ok && items.next(x)) {
      // this CTA's weight rows: 128 plain ones, or 64 gate and 64 up rows
      const int f0 = kGated ? x.ft * 128 + 64 * static_cast<int>(rank)
                            : x.ft * 256 + 128 * static_cast<int>(rank);
      const int wrow = x.e * N + f0;
      const int half = x.width / 2;
      const int xrow = x.p0 + static_cast<int>(rank) * half;
      // more than 48 rows come as one 104-row box (the rows past `half` are not used), fewer
      // in boxes of 16
      const bool tall = half > 48;
      const int boxes = (half + 15) / 16;
      const uint32_t xbytes = tall ? kBBytes : static_cast<uint32_t>(boxes) * 16 * BL;
      const int xt0 = x.p0 / 128;
      const uint32_t sfb_bytes = static_cast<uint32_t>((x.p0 + x.width - 1) / 128 - xt0 + 1) * 512;
      const uint8_t* wsf = args.ws + (c0 * a_tiles + wrow / 128) * 512;
      const uint8_t* wsf_up = args.ws + (c0 * a_tiles + (wrow + F) / 128) * 512;
      const uint8_t* xsf = args.xs + (c0 * b_tiles + xt0) * 512;
      for (int c = c0; c < c1; ++c) {
        if (!__all_sync(0xffffffffu, mbar_wait(bar_empty(stage), phase ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        const uint32_t fb = full0_leader + 8u * stage;  // the even CTA's full barrier
        const uint32_t sa = sbase + stage * kStageBytes;
        const uint32_t sfbar = bar_sf_full(stage);
        const uint32_t ssf = sbase + kOffSf + stage * kSfStage;
        if (issue) {
          if (leader) mbar_arrive_expect_tx(bar_full(stage), 2 * (kABytes + xbytes));
          mbar_arrive_expect_tx(sfbar, (kGated ? 1024u : 512u) + sfb_bytes);
          bulk_load(ssf, wsf, 512, sfbar);
          if constexpr (kGated) bulk_load(ssf + 512, wsf_up, 512, sfbar);
          bulk_load(ssf + kSfA, xsf, sfb_bytes, sfbar);
          if constexpr (kGated) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              tma_load_2d_pair(sa + b * 4096, &args.tm_w, c * BL, wrow + 16 * b, fb);
              tma_load_2d_pair(sa + b * 4096 + 2048, &args.tm_w, c * BL, wrow + F + 16 * b, fb);
            }
          } else {
            tma_load_2d_pair(sa, &args.tm_w, c * BL, wrow, fb);
          }
          if (tall) {
            tma_load_2d_pair(sa + kABytes, &args.tm_x, c * BL, xrow, fb);
          } else {
            for (int b = 0; b < boxes; ++b)
              tma_load_2d_pair(sa + kABytes + b * 2048, &args.tm_x16, c * BL, xrow + 16 * b, fb);
          }
        }
        wsf += a_tiles * 512;
        wsf_up += a_tiles * 512;
        xsf += b_tiles * 512;
        ++chunks;
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
    }
    if (!ok && lane == 0) abort_both();
    // Every stage this CTA filled is released by the MMAs that read it (or, after an abort,
    // the wait gives up after its time limit, long after any copy has landed).
    const uint32_t filled = chunks < kStages ? chunks : kStages;
    for (uint32_t i = 0; i < filled; ++i) {
      const uint32_t c = chunks - 1 - i;
      mbar_wait_drain(bar_empty(static_cast<int>(c % kStages)), (c / kStages) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------- MMA issuer (even CTA only)
    if (leader) {
      const bool issue = elect_one();
      int stage = 0, n = 0;
      uint32_t phase = 0;
      bool ok = true;
      const uint16_t both = static_cast<uint16_t>(0x3u << even);
      const uint64_t a_desc0 = sdesc_kmajor_sw128(sbase);
      Item x;
      while (ok && items.next(x)) {
        const int buf = n & 1;
        if (!__all_sync(0xffffffffu, mbar_wait(bar_acc_empty(buf), ((n >> 1) & 1) ^ 1u, abort_flag))) {
          ok = false;
          break;
        }
        ++n;
        const uint32_t d = tmem + static_cast<uint32_t>(buf * kW);
        const uint32_t idesc = idesc_mxf8_e4m3(256, x.width, 0, 0);
        for (int c = c0; c < c1; ++c) {
          // operands in both CTAs' shared memory, scale factors in both CTAs' TMEM
          if (!__all_sync(0xffffffffu, mbar_wait(bar_full(stage), phase, abort_flag))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tsf = tmem + kSfCol0 + 16u * stage;
          const uint64_t ad = a_desc0 + static_cast<uint32_t>(stage * (kStageBytes >> 4));
          const uint64_t bd = ad + (kABytes >> 4);
          if (issue) {
#pragma unroll
            for (uint32_t kb = 0; kb < 4; ++kb)
              mma_mxf8_block32_pair(d, ad + 2 * kb, bd + 2 * kb, idesc | (kb << 4) | (kb << 29), tsf,
                                    tsf + 8, (c - c0) != 0 || kb != 0);
            mma_commit_pair(bar_empty(stage), both);
          }
          __syncwarp();
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        if (issue) mma_commit_pair(bar_acc_full(buf), both);
        __syncwarp();
      }
      if (!ok && lane == 0) abort_both();
      // All MMAs issued by this warp's lane complete before TMEM is released.
      if (issue) {
        mma_commit_pair(bar_done, static_cast<uint16_t>(0x1u << even));
        mbar_wait_drain(bar_done, 0);
      }
      __syncwarp();
    }
  } else if (warp >= kSfWarp0) {
    // ----------------------------------- scale writers: TMEM lane quarter warp % 4
    // tcgen05.mma reads the scale of operand row j from lane j % 32, column j / 32 of every
    // lane quarter, one byte per 32-element block.
    const uint32_t quarter = static_cast<uint32_t>(warp & 3);
    const uint32_t full0_leader = map_to_cta(bar_full(0), even);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    Item x;
    while (ok && items.next(x)) {
      // Row p0 + 32 q + lane of x is word (shift + q) of this lane's row of the atoms: 16 bytes
      // per atom hold the four rows r0, r0 + 32, r0 + 64, r0 + 96.
      const uint32_t start = static_cast<uint32_t>(x.p0 & 127) + lane;
      const uint32_t r0 = start & 31u, shift = start >> 5;
      const bool by1 = shift & 1u, by2 = shift & 2u, by4 = shift & 4u;
      for (int c = c0; c < c1; ++c) {
        const int st = stage;
        if (!__all_sync(0xffffffffu, mbar_wait(bar_sf_full(st), phase, abort_flag))) {
          ok = false;
          break;
        }
        const uint32_t ssf = sbase + kOffSf + st * kSfStage;
        uint32_t a[4], b[12];
        if constexpr (kGated) {
          // tile row 32 r1 + lane is row 64 rank + 16 r1 + lane % 16 of the gate (up) atom
          const uint32_t src = ssf + (lane >> 4) * 512u + (lane & 15u) * 16u + rank * 8u;
          const uint2 even = ld_shared_v2(src), odd = ld_shared_v2(src + 256u);
          a[0] = even.x, a[1] = odd.x, a[2] = even.y, a[3] = odd.y;
        } else {
          const uint4 v = ld_shared_v4(ssf + 16u * lane);
          a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
        }
#pragma unroll
        for (int j = 0; j < 3; ++j) {
          const uint4 v = ld_shared_v4(ssf + kSfA + 512u * j + 16u * r0);
          b[4 * j] = v.x, b[4 * j + 1] = v.y, b[4 * j + 2] = v.z, b[4 * j + 3] = v.w;
        }
        // seven words from `shift` (0 .. 4) on; the eighth column is not read by the MMA
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = by4 ? b[j + 4] : b[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = by2 ? b[j + 2] : b[j];
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] = by1 ? b[j + 1] : b[j];
        const uint32_t tsf = tmem + (quarter * 32u << 16) + kSfCol0 + 16u * st;
        tmem_st_x4(tsf, a);
        tmem_st_x8(tsf + 8, *reinterpret_cast<uint32_t(*)[8]>(&b[0]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(full0_leader + 8u * st);
        if (++stage == kStages) stage = 0, phase ^= 1u;
      }
    }
    if (!ok && lane == 0) abort_both();
  } else {
    // ------------------------------------------------------------ epilogue
    const int ew = warp - 2;
    const int quarter = warp & 3;  // TMEM lanes this warp may access
    const int part = ew >> 2;      // every kEpiParts-th 16-column group
    const uint32_t acc_empty0 = map_to_cta(bar_acc_empty(0), even);
    const uint32_t tile = sbase + kOffTurn + static_cast<uint32_t>(ew) * kTurnBytes;
    constexpr int kCh = kGated ? 2 : 4;  // 16-byte chunks of y per row and warp
    const uint32_t frag = tile + Turn<kCh>::fragment(), piece = tile + Turn<kCh>::piece();
    const __nv_bfloat16* res = static_cast<const __nv_bfloat16*>(args.residual);
    const bool save = args.z != nullptr;
    // Partial accumulators in the ring: 2 KB per (pair, 16-column group, lane quarter).
    auto partial_at = [&](int j, int g) {
      return sbase + static_cast<uint32_t>(((j - 1) * (kSplitRows / 16) + g) * 4 + quarter) * 2048u + lane * 16u;
    };
    if constexpr (S > 1) {
      bool send = false;
      Item x;
      if (split > 0 && items.next(x)) {
        send = __all_sync(0xffffffffu, mbar_wait(bar_acc_full(0), 0, abort_flag));
        if (!send && lane == 0) abort_both();
      }
      tc_fence_after();
      cluster_sync();  // every pair's MMAs have ended: the first pair's ring is free
      if (send) {
        for (int g = part; g * 16 < x.nrows; g += kEpiParts) {
          uint32_t r[16];
          tmem_ld_16x256b_x2(tmem + (static_cast<uint32_t>(quarter * 32) << 16) + 16u * g, r);
          tmem_ld_16x256b_x2(tmem + (static_cast<uint32_t>(quarter * 32 + 16) << 16) + 16u * g, r + 8);
          tmem_wait_ld_regs(r);
          const uint32_t to = map_to_cta(partial_at(split, g), rank);
#pragma unroll
          for (int i = 0; i < 4; ++i) st_cluster_v4(to + 512u * i, r + 4 * i);
        }
      }
      cluster_sync();  // the partial accumulators are there
    }
    // The warp's first group of an item moves on by one from item to item: 13 groups over three
    // warps are then 13 each after three items, not 15, 12 and 12, as a warp may run one item ahead
    // of the others (65536 rows of 16 experts, K = 256: 1024 columns with GELU and saved
    // pre-activation 73 to 81 us from process to process, with a fixed first group 79; 2048
    // columns with SwiGLU 67 against 71).
    int n = 0, first = part;
    Item x;
    while (split == 0 && items.next(x)) {
      // the warp's first column of y; of z too (gated: gate columns, up columns F further)
      const int col = kGated ? x.ft * 128 + 64 * static_cast<int>(rank) + 16 * quarter
                             : x.ft * 256 + 128 * static_cast<int>(rank) + 32 * quarter;
      // bias[h][i]: z column of lane 16 h + 8 i + lane_id / 4
      float bias[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          bias[h][i] = args.bias == nullptr
                           ? 0.0f
                           : args.bias[static_cast<size_t>(x.e) * N + col + h * (kGated ? F : 16) +
                                       8 * i + static_cast<int>(lane >> 2)];
      const int buf = n & 1;
      if (!__all_sync(0xffffffffu, mbar_wait(bar_acc_full(buf), (n >> 1) & 1, abort_flag))) {
        if (lane == 0) abort_both();
        break;
      }
      ++n;
      tc_fence_after();
      const uint32_t ta = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(buf * kW);
      uint32_t r[16];
      if (first * 16 < x.nrows) {
        tmem_ld_16x256b_x2(ta + 16u * first, r);
        tmem_ld_16x256b_x2(ta + (16u << 16) + 16u * first, r + 8);
      }
      // this lane's pieces of its first group's rows; a step takes it to the warp's next group
      const size_t row = static_cast<size_t>(x.row0) + 16 * first + Turn<kCh>::row();
      const size_t pitch_y = F, pitch_z = N;
      __nv_bfloat16* yp = static_cast<__nv_bfloat16*>(args.y) + row * pitch_y + col + Turn<kCh>::col();
      __nv_bfloat16* zp = static_cast<__nv_bfloat16*>(args.z) + row * pitch_z + col + Turn<kCh>::col();
      const __nv_bfloat16* rp = res + row * pitch_y + col + Turn<kCh>::col();
      uint4 rv[kCh / 2];
      if (res != nullptr && first * 16 < x.nrows) Turn<kCh>::load(rp, pitch_y, x.nrows - 16 * first, rv);
      for (int g = first; g * 16 < x.nrows; g += kEpiParts) {
        const int left = x.nrows - 16 * g;  // rows of this group that exist
        const bool more = (g + kEpiParts) * 16 < x.nrows;
        tmem_wait_ld_regs(r);
        // z[h][b][j]: lane 16 h + 8 (j / 2) + lane_id / 4, row 8 b + 2 (lane_id % 4) + j % 2
        float z[2][2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              z[h][b][j] = __uint_as_float(r[8 * h + 4 * b + j]);
              if constexpr (S == 1) z[h][b][j] += bias[h][j >> 1];
            }
        if constexpr (S > 1) {
#pragma unroll
          for (int k = 1; k < S; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 v = ld_shared_v4(partial_at(k, g) + 512u * i);
              z[i >> 1][i & 1][0] += __uint_as_float(v.x);
              z[i >> 1][i & 1][1] += __uint_as_float(v.y);
              z[i >> 1][i & 1][2] += __uint_as_float(v.z);
              z[i >> 1][i & 1][3] += __uint_as_float(v.w);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) z[i >> 1][i & 1][j] += bias[i >> 1][j >> 1];
        }
        if (more) {
          tmem_ld_16x256b_x2(ta + 16u * (g + kEpiParts), r);
          tmem_ld_16x256b_x2(ta + (16u << 16) + 16u * (g + kEpiParts), r + 8);
        }
        uint32_t f[8], rf[8];
        __syncwarp();  // the previous group has left the staging tile
        if (res != nullptr) {
          Turn<kCh>::fill(piece, rv);
          rp += 16 * kEpiParts * pitch_y;
          if (more) Turn<kCh>::load(rp, pitch_y, left - 16 * kEpiParts, rv);
          __syncwarp();
          Turn<kCh>::get(frag, rf);
          __syncwarp();
        }
        if (save) {
          if constexpr (kGated) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int i = 0; i < 2; ++i) f[2 * b + i] = pack_bf16(z[h][b][2 * i], z[h][b][2 * i + 1]);
              Turn<2>::put(frag + h * 512, f);
            }
          } else {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                f[4 * b + i] = pack_bf16(z[i >> 1][b][2 * (i & 1)], z[i >> 1][b][2 * (i & 1) + 1]);
            Turn<4>::put(frag, f);
          }
          __syncwarp();
          if constexpr (kGated) {
            Turn<2>::store(piece, zp, pitch_z, left);
            Turn<2>::store(piece + 512, zp + F, pitch_z, left);
          } else {
            Turn<4>::store(piece, zp, pitch_z, left);
          }
          zp += 16 * kEpiParts * pitch_z;
        }
        // y in z's place: [0][b][j] when gated
#pragma unroll
        for (int h = 0; h < (kGated ? 1 : 2); ++h)
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              act_value2<kInner>(z[h][b][j], z[h][b][j + 1]);
              if constexpr (kGated) {
                z[h][b][j] *= z[1][b][j];
                z[h][b][j + 1] *= z[1][b][j + 1];
              }
            }
        if (res != nullptr) {
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < kCh; ++i) {
              const float2 v = unpack_bf16(rf[kCh * b + i]);
              z[i >> 1][b][2 * (i & 1)] += v.x;
              z[i >> 1][b][2 * (i & 1) + 1] += v.y;
            }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < kCh; ++i)
            f[kCh * b + i] = pack_bf16(z[i >> 1][b][2 * (i & 1)], z[i >> 1][b][2 * (i & 1) + 1]);
        __syncwarp();  // z has left the tile
        Turn<kCh>::put(frag, f);
        __syncwarp();
        Turn<kCh>::store(piece, yp, pitch_y, left);
        yp += 16 * kEpiParts * pitch_y;
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(acc_empty0 + 8u * buf);
      first = first + 1 == kEpiParts ? 0 : first + 1;
    }
  }

  if constexpr (S > 1) {
    if (warp < 2 || warp >= kSfWarp0) {  // the epilogue's two barriers
      __syncwarp();
      cluster_sync();
      cluster_sync();
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // no pair MMA reads this CTA's shared memory or writes its TMEM any more
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

template <int ACT, int S>
cudaLaunchConfig_t split_config(size_t smem, long long clusters, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * 2 * S));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  attr->id = cudaLaunchAttributeClusterDimension;
  attr->val.clusterDim.x = 2 * S;
  attr->val.clusterDim.y = 1;
  attr->val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <int ACT, int S>
cudaError_t set_smem() {
  static thread_local uint64_t attr_ctx = 0;
  return set_smem_attr_once(reinterpret_cast<const void*>(grouped_act_kernel<ACT, S>),
                            act_smem_bytes(kMaxExperts), &attr_ctx);
}

// Clusters of S pairs that the current context runs at once: none where a process has a share of
// the SMs that is too small.  Asked once per context and thread.
template <int ACT, int S>
int clusters_at_once() {
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int active = 0;
  if (asked_ctx != 0 && asked_ctx == current_context_id()) return active;
  if (set_smem<ACT, S>() != cudaSuccess) return 0;
  cudaLaunchAttribute attr = {};
  const cudaLaunchConfig_t cfg = split_config<ACT, S>(act_smem_bytes(kMaxExperts), 1, &attr);
  if (cudaOccupancyMaxActiveClusters(&active, grouped_act_kernel<ACT, S>, &cfg) != cudaSuccess) {
    (void)cudaGetLastError();  // a size that does not fit is no error of the call
    active = 0;
  }
  asked_ctx = current_context_id();
  return active;
}

template <int ACT, int S>
cudaError_t launch_split(const ActMmArgs& a, long long clusters, cudaStream_t stream) {
  const cudaError_t err = set_smem<ACT, S>();
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr = {};
  cudaLaunchConfig_t cfg = split_config<ACT, S>(act_smem_bytes(a.E), clusters, &attr);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, grouped_act_kernel<ACT, S>, a);
}

template <int ACT>
cudaError_t launch(const ActMmArgs& a, int num_sms, cudaStream_t stream) {
  // The exact number of row tiles is known on the device only.
  const long long experts = a.M < a.E ? a.M : a.E;
  long long items = (static_cast<long long>(a.M) / kW + experts) * (a.N / 256);
  if (items < 1) items = 1;
  // Few rows and items: split the contraction over clusters of four or two pairs, as long as
  // these run at once (the device takes 15 clusters of 8 CTAs or 36 of 4; a 16th cluster of 8
  // waits for a whole one and costs 9 us).  16 rows of one expert, launch included: 1024 x 16384
  // 36 us with one pair an item, 26 with two, 20 with four; 1024 x 4096 18, 16 and 15 us.
  const int nch = a.K / BL;
  const int most = a.max_cluster > 0 ? a.max_cluster : 8;
  if (a.M <= kSplitRows && nch >= 8 && items * 8 <= num_sms * 4 / 5 && most >= 8 &&
      items <= clusters_at_once<ACT, 4>())
    return launch_split<ACT, 4>(a, items, stream);
  if (a.M <= kSplitRows && nch >= 4 && items * 4 <= num_sms * 15 / 16 && most >= 4 &&
      items <= clusters_at_once<ACT, 2>())
    return launch_split<ACT, 2>(a, items, stream);
  const long long pairs = items < num_sms / 2 ? items : num_sms / 2;  // at most one per item
  return launch_split<ACT, 1>(a, pairs, stream);
}

}  // namespace

int act_row_box() { return kW / 2; }

cudaError_t launch_grouped_act(const ActMmArgs& a, int act, int num_sms, cudaStream_t stream) {
  switch (act) {
    case kActNone: return launch<kActNone>(a, num_sms, stream);
    case kActRelu: return launch<kActRelu>(a, num_sms, stream);
    case kActGelu: return launch<kActGelu>(a, num_sms, stream);
    case kActSilu: return launch<kActSilu>(a, num_sms, stream);
    case kActSwiglu: return launch<kActSwiglu>(a, num_sms, stream);
    case kActGeglu: return launch<kActGeglu>(a, num_sms, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace mgw
