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
// HBM bounds it: the input once, base and out once, the adapters from L2.  16384 rows of one adapter,
// 4096 x 4096, rank 64, u saved: 75 us, 5.4 TB/s; of these 25 us the input's half (a bare TMA read of the
// same boxes takes 24.5), 36 the output's (half of its traffic is writes), the rest launch, setup and
// the exchange between the halves, when HBM is idle.  65536 gathered rows of 64 adapters, 4096 x 1536,
// rank 32 (every row of x is read eight times): 135 us, with HBM at 49% and L2 at 35% of their peaks: what
// bounds it are the loads that two CTAs an SM have in flight in either half.
//
// Both halves stream through one ring of shared-memory slots: 64 columns of 128 rows (the input's,
// then the base's, which become the output's in place) and the weight's tile that goes with them.
// Roles: warp 0 loads by TMA, warp 1 issues the MMAs, warps 2-5 (where one CTA fills an SM, 6-9 too, a
// second set) have a TMEM lane quarter each.  They copy the input's rows where these are few or lie apart (16 bytes a
// lane; gathered by TMA, four rows an instruction, 65536 rows took 236 us in all instead of 159), turn the
// partial sums into the intermediate, and take the output's tiles in turns: accumulator + base, rounded
// once, stored by TMA, or as whole 128-byte row pieces where rows lie apart.
#include <cuda_runtime.h>

#include <cstdint>

#include "lora.cuh"

namespace mgw {
namespace {

using namespace lora;

constexpr int kRows = 128;
constexpr int kBk = 64;               // columns per slot, of the input and of the output
constexpr int kXBytes = kRows * 128;  // 128 rows of 64 bf16
constexpr int kMaxSlots = 12;
constexpr int kBufs = 4;              // accumulators of 64 columns
constexpr uint32_t kTmemCols = 256;   // those; before them the partial sums
constexpr int kBars = 4 * kMaxSlots + 1 + 2 * kBufs + 1;
constexpr int kTmpBytes = 96;         // find_tile's ints (18 of ten warps, the most); then [4] TMEM [5] abort

// Epilogue sets of four warps: two where one CTA fills an SM, one where two CTAs share it.  (Two CTAs of
// two sets have 80 registers a thread; what did not fit, which no L1 holds beside this much shared
// memory, made the output's half 1.6 times as long.)  Registers are given out to four warps at a time.
constexpr int kManySets = 2;
constexpr int threads_of(int sets) { return 64 + 128 * sets; }
constexpr int bound_of(int sets) { return (threads_of(sets) + 127) / 128 * 128; }

// RQ: the rank, rounded up to 32, 64 or 128.  The intermediate's two parts are 2 RQ columns, in
// 64-wide tiles.  The ring's slots are as large as the tile's rows and the rank need, so that few rows
// have all their loads on the way at once; the tensor core reads 128 rows all the same, into the
// slots behind (those rows' results go nowhere).
template <int RQ>
struct Plan {
  static constexpr int kWBytes = RQ == 128 ? 16384 : 8192;  // of a slot, at most
  static constexpr int kU = RQ * 512;
  // Partial sums are kept in this many accumulators in turn, added up at the end: the tensor core
  // cuts each addition's low bits off, always downwards, so a long chain drifts (u of K = 4096: 4.4e-6
  // relative in one chain, 4.7e-7 in four).
  static constexpr int kChains = RQ == 128 ? 2 : 4;
  // The ring: two CTAs an SM, or one with a long ring where there are few.
  static constexpr int kShort = (RQ == 128 ? 160 : (RQ == 64 ? 78 : 94)) * 1024;
  static constexpr int kLong = (RQ == 128 ? 160 : (RQ == 64 ? 192 : 208)) * 1024;
  static constexpr size_t smem(int ring) {
    return static_cast<size_t>(ring) + kU + kBars * 8 + kTmpBytes + kRows * 4 + 1024;
  }
  // the CTAs' partial sums lie at the ring's end while they are exchanged; two slots remain
  static_assert(kShort - RQ * 512 >= kXBytes + kWBytes && kXBytes <= kU, "ring");
};
static_assert(2 * (Plan<32>::smem(Plan<32>::kShort) + 1024) <= 228 * 1024 &&
                  2 * (Plan<64>::smem(Plan<64>::kShort) + 1024) <= 228 * 1024 &&
                  Plan<32>::smem(Plan<32>::kLong) <= 227 * 1024 && Plan<64>::smem(Plan<64>::kLong) <= 227 * 1024 &&
                  Plan<128>::smem(Plan<128>::kLong) <= 227 * 1024,
              "shared memory budget");
static_assert(kBars * 8 % 16 == 0, "alignment");

// A place in a ring of n: its slot and the parity of its round.
struct Turn {
  int slot;
  uint32_t phase;
  __device__ __forceinline__ void step(int by, int n) {
    slot += by;
    if (slot >= n) slot -= n, phase ^= 1u;
  }
};

template <bool TRANS, int RQ, int SETS>
__global__ void __launch_bounds__(bound_of(SETS), SETS == 1 ? 2 : 1) lora_kernel(const __grid_constant__ LoraArgs a) {
  using P = Plan<RQ>;
  constexpr int G = P::kChains, kThreads = threads_of(SETS);
  constexpr int COPY = SETS < 2 ? SETS : 2;  // sets that copy the input's rows
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t su = sbase + a.ring;  // the intermediate
  const uint32_t bar0 = su + P::kU;
  uint8_t* misc = smem + a.ring + P::kU + kBars * 8;
  int* s_tmp = reinterpret_cast<int*>(misc);                          // find_tile; [4] TMEM [5] abort
  int* s_rows = reinterpret_cast<int*>(misc + kTmpBytes);                    // place of the 128 output rows
  volatile int* abort_flag = reinterpret_cast<volatile int*>(s_tmp + 5);
  const int tid = threadIdx.x, warp = tid >> 5;
  const uint32_t lane = lane_id();
  const int C = a.cluster;
  const int rank = C > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  if (tid == 0) {
    tma_prefetch_desc(&a.tm_x);
    tma_prefetch_desc(&a.tm_w1);
    tma_prefetch_desc(&a.tm_w2);
  }
  wait_for_launch_before();

  RowTile t;
  if (!find_tile<kThreads, kRows>(a.off, a.E, a.M, static_cast<int>(blockIdx.x) / C, s_tmp, a.status, t)) return;
  if (t.nrows == 0) return;
  const int N = a.N;
  const int ntiles = (N + kBk - 1) / kBk;
  const int nt0 = static_cast<int>(static_cast<long long>(ntiles) * rank / C);
  __nv_bfloat16* out = static_cast<__nv_bfloat16*>(a.out);
  const __nv_bfloat16* base = static_cast<const __nv_bfloat16*>(a.base);
  const int nt1 = out == nullptr ? nt0 : static_cast<int>(static_cast<long long>(ntiles) * (rank + 1) / C);

  if (t.e == a.E) {
    // Rows without an adapter: their base, or zeros.  All rows' places first, then 16 bytes a thread and
    // step, four steps on their way.
    if (a.u != nullptr && rank == 0)
      for (int i = tid; i < t.nrows * a.R; i += kThreads) a.u[static_cast<size_t>(t.row0) * a.R + i] = 0.0f;
    const int wide = min(nt1 * kBk, N) / 8 - nt0 * (kBk / 8);  // 16-byte pieces of a row
    // (looked at even where nothing is copied: an index out of range is reported)
    for (int i = tid; i < t.nrows; i += kThreads)
      s_rows[i] = row_place(a.out_index, t.row0 + i, a.out_rows, rank == 0 ? a.status : nullptr);
    if (out == nullptr || out == base || wide <= 0) return;
    __syncthreads();
    constexpr int kSteps = 4;
    for (int i0 = tid; i0 < t.nrows * wide; i0 += kSteps * kThreads) {
      uint4 v[kSteps];
      size_t at[kSteps];
      bool there[kSteps];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int i = i0 + k * kThreads;
        const int o = i < t.nrows * wide ? s_rows[i / wide] : -1;
        there[k] = o >= 0;
        at[k] = static_cast<size_t>(max(o, 0)) * N + nt0 * kBk + i % wide * 8;
        v[k] = make_uint4(0u, 0u, 0u, 0u);
        if (base != nullptr && there[k]) v[k] = *reinterpret_cast<const uint4*>(base + at[k]);
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        if (there[k]) *reinterpret_cast<uint4*>(out + at[k]) = v[k];
    }
    return;
  }

  // Rows in order come as one box, a tile's last rows too as long as they are many: the rows behind
  // them, another adapter's, meet nothing of this one's.  Others are copied.
  const bool many = t.nrows >= kRows / 2;
  const bool in_box = a.in_index == nullptr && many, out_box = a.out_index == nullptr && many;
  const bool copy_base = base != nullptr && !out_box;
  const int RP = (a.R + 15) & ~15;
  const int rows8 = many ? kRows : (t.nrows + 7) & ~7;
  const int x_tile = rows8 * 128;  // bytes of a slot's rows; the weight's tile lies behind them
  const int w1_tile = TRANS ? P::kWBytes : RP * 128, w2_tile = TRANS ? RP * 128 : P::kWBytes;
  const int slot1 = x_tile + w1_tile, slot2 = x_tile + w2_tile;
  const int S1 = min(kMaxSlots, a.ring / slot1), S2 = min(kMaxSlots, a.ring / slot2);
  const int part_at = a.ring - rows8 * RP * 4;
  const uint32_t part = sbase + part_at;  // partial sums
  // Slots of the output's half that may be filled while the partial sums are exchanged.
  const int early = C > 1 ? min(S2, part_at / slot2) : S2;
  const int nch = (a.K + kBk - 1) / kBk;
  const int c0 = static_cast<int>(static_cast<long long>(nch) * rank / C);
  const int c1 = static_cast<int>(static_cast<long long>(nch) * (rank + 1) / C);
  const int chunks = c1 - c0, tiles = nt1 - nt0;

  auto bar_full = [&](int s) { return bar0 + 8u * s; };
  auto bar_empty = [&](int s) { return bar0 + 8u * (kMaxSlots + s); };
  auto bar_bfull = [&](int s) { return bar0 + 8u * (2 * kMaxSlots + s); };
  auto bar_bempty = [&](int s) { return bar0 + 8u * (3 * kMaxSlots + s); };
  const uint32_t bar_sum = bar0 + 8u * (4 * kMaxSlots);
  auto bar_acc = [&](int s) { return bar0 + 8u * (4 * kMaxSlots + 1 + s); };
  auto bar_free = [&](int s) { return bar0 + 8u * (4 * kMaxSlots + 1 + kBufs + s); };
  const uint32_t bar_done = bar0 + 8u * (4 * kMaxSlots + 1 + 2 * kBufs);
  if (tid < kMaxSlots) {
    mbar_init(bar_full(tid), in_box ? 1 : 1 + 128 * COPY);
    mbar_init(bar_empty(tid), 1);
    mbar_init(bar_bfull(tid), 1);
    mbar_init(bar_bempty(tid), 4);
    if (tid < kBufs) {
      mbar_init(bar_acc(tid), 1);
      mbar_init(bar_free(tid), 4);
    }
    if (tid == 0) {
      mbar_init(bar_sum, 1);
      mbar_init(bar_done, 1);
      s_tmp[5] = 0;
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(s_tmp + 4), kTmemCols);
    tmem_relinquish();
  }
  if (tid >= 64 && tid < 64 + kRows) {
    const int i = tid - 64;
    s_rows[i] = i < t.nrows ? row_place(a.out_index, t.row0 + i, a.out_rows, rank == 0 ? a.status : nullptr) : -1;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(s_tmp[4]);
  bool ok = true;
  // the gradients' launch may start as soon as it finds room; it waits for this one's blocks itself
  if constexpr (TRANS) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Turn in = {0, 0};
    int n = 0;
    for (int c = c0; c < c1; ++c) {
      ok = wait_all(bar_empty(in.slot), in.phase ^ 1u, abort_flag);
      if (!ok) break;
      if (lane == 0) {
        const uint32_t fb = bar_full(in.slot), sx = sbase + in.slot * slot1, sw = sx + x_tile;
        mbar_arrive_expect_tx(fb, (in_box ? static_cast<uint32_t>(kXBytes) : 0u) + w1_tile);
        if constexpr (TRANS) {
#pragma unroll
          for (int b = 0; b < P::kWBytes / 8192; ++b) tma_load_3d(sw + b * 8192, &a.tm_w1, 64 * b, c * kBk, t.e, fb);
        } else {
          tma_load_3d(sw, &a.tm_w1, c * kBk, 0, t.e, fb);
        }
        if (in_box) tma_load_2d(sx, &a.tm_x, c * kBk, t.row0, fb);
      }
      __syncwarp();
      ++n;
      in.step(1, S1);
    }
    // Behind the last MMA that reads them the slots serve the output's half.
    ok = ok && wait_all(bar_sum, 0, abort_flag);
    const bool base_box = base != nullptr && out_box;
    Turn to = {0, 0};
    int i = 0;
    auto load_tile = [&]() {
      if (lane == 0) {
        const uint32_t fb = bar_bfull(to.slot), dst = sbase + to.slot * slot2, sw = dst + x_tile;
        const int col = (nt0 + i) * kBk;
        mbar_arrive_expect_tx(fb, (base_box ? static_cast<uint32_t>(kXBytes) : 0u) + w2_tile);
        if (base_box) tma_load_2d(dst, &a.tm_base, col, t.row0, fb);
        if constexpr (TRANS) {
          tma_load_3d(sw, &a.tm_w2, col, 0, t.e, fb);
        } else {
#pragma unroll
          for (int b = 0; b < P::kWBytes / 8192; ++b) tma_load_3d(sw + b * 8192, &a.tm_w2, 64 * b, col, t.e, fb);
        }
      }
      __syncwarp();
      ++i;
      to.step(1, S2);
    };
    cluster_arrive();
    while (ok && i < tiles && i < early) load_tile();
    cluster_wait();  // partial sums are there
    cluster_sync();  // the intermediate is
    fence_async_all();
    while (ok && i < tiles) {
      ok = wait_all(bar_bempty(to.slot), to.phase ^ 1u, abort_flag);
      if (ok) load_tile();
    }
    if (!ok && lane == 0) give_up(abort_flag, a.status);
    // Never leave the CTA with copies still landing in shared memory (behind a wait that ran out they
    // have long landed).
    bool landed = true;
    for (int k = n > S1 ? n - S1 : 0; landed && k < n; ++k) landed = mbar_wait_drain(bar_full(k % S1), (k / S1) & 1u);
    for (int k = i > S2 ? i - S2 : 0; landed && k < i; ++k) landed = mbar_wait_drain(bar_bfull(k % S2), (k / S2) & 1u);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const bool issue = elect_one();
    {
      const uint32_t idesc = idesc_bf16(RP, false, TRANS);
      Turn in = {0, 0};
      for (int i = 0; i < chunks; ++i) {
        ok = wait_all(bar_full(in.slot), in.phase, abort_flag);
        if (!ok) break;
        if (!in_box) fence_async_smem();  // the copies are generic writes
        tc_fence_after();
        const uint32_t sx = sbase + in.slot * slot1, sw = sx + x_tile;
        const uint64_t ad = sdesc_kmajor_sw128(sx);
        const uint64_t bd = TRANS ? sdesc_mn_sw128(sw, 8192) : sdesc_kmajor_sw128(sw);
        const uint32_t d = tmem + static_cast<uint32_t>(i % G * RP);
        if (issue) {
#pragma unroll
          for (uint32_t k = 0; k < kBk / 16; ++k)
            mma_bf16(d, ad + kStepK * k, bd + (TRANS ? kStepMn : kStepK) * k, idesc, i >= G || k != 0);
          mma_commit(bar_empty(in.slot));
        }
        __syncwarp();
        in.step(1, S1);
      }
      if (issue) mma_commit(bar_sum);
      __syncwarp();
    }
    cluster_sync();
    cluster_sync();
    tc_fence_after();
    fence_async_all();
    const uint32_t idesc = idesc_bf16(kBk, false, TRANS);
    Turn to = {0, 0}, acc = {0, 0};
    for (int i = 0; ok && i < tiles; ++i) {
      ok = wait_all(bar_bfull(to.slot), to.phase, abort_flag) &&
           wait_all(bar_free(acc.slot), acc.phase ^ 1u, abort_flag);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sw = sbase + to.slot * slot2 + x_tile;
      const uint32_t d = tmem + static_cast<uint32_t>(acc.slot * kBk);
      if (issue) {
        for (int p = 0; p < 2; ++p) {
          for (int k = 0; k < RP / 16; ++k) {
            const int col = p * RQ + 16 * k;  // of the intermediate's two parts
            const uint64_t ad = sdesc_kmajor_sw128(su + (col >> 6) * kXBytes) + kStepK * ((col & 63) >> 4);
            const uint64_t bd = TRANS ? sdesc_mn_sw128(sw, 8192) + kStepMn * k
                                      : sdesc_kmajor_sw128(sw + (k >> 2) * 8192) + kStepK * (k & 3);
            mma_bf16(d, ad, bd, idesc, p != 0 || k != 0);
          }
        }
        mma_commit(bar_acc(acc.slot));
      }
      __syncwarp();
      to.step(1, S2);
      acc.step(1, kBufs);
    }
    if (!ok && lane == 0) give_up(abort_flag, a.status);
    if (issue) {
      mma_commit(bar_done);
      mbar_wait_drain(bar_done, 0);
    }
    __syncwarp();
  } else {
    const int ew = warp - 2, quarter = warp & 3, set = ew >> 2;
    const int sub = static_cast<int>(lane >> 3), ch = static_cast<int>(lane & 7);
    const float scale = a.scale != nullptr ? a.scale[t.e] : 1.0f;
    if (!in_box && set < COPY) {
      // ------------------------------------------- the input's rows: eight lanes a row
      // Rows behind the tile's last stay as they are: whatever they hold goes into rows that nobody
      // stores.
      constexpr int kMine = 8 / COPY;  // times four rows a warp
      const __nv_bfloat16* src[kMine];
      uint32_t dst[kMine];
      bool there[kMine];
      int live = 0;
#pragma unroll
      for (int p = 0; p < kMine; ++p) {
        const int r = 4 * kMine * ew + 4 * p + sub;
        int o = -1;
        if (r < t.nrows)
          o = row_place(a.in_index, t.row0 + r, a.in_rows, rank == 0 && ch == 0 ? a.status : nullptr), ++live;
        there[p] = o >= 0;
        src[p] = static_cast<const __nv_bfloat16*>(a.in) + static_cast<size_t>(max(o, 0)) * a.K + 8 * ch;
        dst[p] = sbase + swz(r, ch);
      }
      Turn in = {0, 0};
      for (int i = 0; i < chunks; ++i) {
        ok = wait_all(bar_empty(in.slot), in.phase ^ 1u, abort_flag);
        if (!ok) break;
        const int col = (c0 + i) * kBk;
        const bool inside = col + 8 * ch < a.K;
#pragma unroll
        for (int p = 0; p < kMine; ++p)
          if (p < live) copy16(dst[p] + in.slot * slot1, src[p] + (inside ? col : -8 * ch), inside && there[p]);
        copy_arrive(bar_full(in.slot));
        in.step(1, S1);
      }
    }
    // Rows of the tile that Q's blocks need (see LoraArgs): they are read up to a multiple of 16.
    const int q_rows = TRANS && a.qv != nullptr ? (t.nrows + 15) & ~15 : t.nrows;
    // Q's blocks, a thread a rank and eight rows; the cluster's CTAs share the rows.
    auto q_piece = [&](uint8_t* q, int octet, int j, int lo) {
      return reinterpret_cast<uint4*>(q + (2 * static_cast<size_t>(static_cast<int>(blockIdx.x) / C) + (octet >> 3)) *
                                              (256u * RP) + lo * RP * 128 + swz(j, octet & 7));
    };
    const int octets = (q_rows / 8 - rank + C - 1) / C;
    if constexpr (TRANS) {
      // u's, while the products run
      if (a.qv != nullptr) {
        for (int i = tid - 64; i < octets * RP; i += 128 * SETS) {
          const int j = i % RP, o = rank + C * (i / RP);
          float f[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int r = 8 * o + k;
            f[k] = r < t.nrows && j < a.R ? scale * a.u_in[static_cast<size_t>(t.row0 + r) * a.R + j] : 0.0f;
          }
          uint4 hi, lo;
          split2(f[0], f[1], hi.x, lo.x);
          split2(f[2], f[3], hi.y, lo.y);
          split2(f[4], f[5], hi.z, lo.z);
          split2(f[6], f[7], hi.w, lo.w);
          *q_piece(a.qu, o, j, 0) = hi;
          *q_piece(a.qu, o, j, 1) = lo;
        }
        __syncwarp();
      }
    }
    // ------------------------------------------- the partial sums
    const uint32_t tq = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
    const int row = quarter * 32 + static_cast<int>(lane);
    ok = wait_all(bar_sum, 0, abort_flag) && ok;
    tc_fence_after();
    // Eight ranks from 8 j8 on of a row: u, and the two parts into the CTAs' intermediates.
    auto finish = [&](int r, int j8, float (&v)[8]) {
      const bool live = r < t.nrows && 8 * j8 < a.R;
      if (live && a.u != nullptr) {
        float4* u = reinterpret_cast<float4*>(a.u + static_cast<size_t>(t.row0 + r) * a.R + 8 * j8);
        u[0] = make_float4(v[0], v[1], v[2], v[3]);
        u[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = live ? v[j] * scale : 0.0f;
      uint4 hi, lo;
      split2(v[0], v[1], hi.x, lo.x);
      split2(v[2], v[3], hi.y, lo.y);
      split2(v[4], v[5], hi.z, lo.z);
      split2(v[6], v[7], hi.w, lo.w);
      const uint32_t hc = 8u * j8, lc = RQ + 8u * j8;
      const uint32_t to_hi = su + (hc >> 6) * kXBytes + swz(r, (hc & 63) >> 3);
      const uint32_t to_lo = su + (lc >> 6) * kXBytes + swz(r, (lc & 63) >> 3);
      if (C == 1) {
        st_shared_u4(to_hi, hi);
        st_shared_u4(to_lo, lo);
      } else {
        for (int p = 0; p < C; ++p) {
          st_cluster_u4(map_to_cta(to_hi, p), hi);
          st_cluster_u4(map_to_cta(to_lo, p), lo);
        }
      }
    };
    const int chains = min(G, chunks);
    for (int j = 16 * set; j < RP; j += 16 * SETS) {
      float v[2][8];
      uint32_t r[G][16];
#pragma unroll
      for (int g = 0; g < G; ++g)
        if (g < chains) tmem_ld_x16(tq + g * RP + j, r[g]);
      tmem_wait_ld();
#pragma unroll
      for (int g = 0; g < G; ++g) tmem_loaded(r[g]);
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        float sum = __uint_as_float(r[0][k]);
#pragma unroll
        for (int g = 1; g < G; ++g)
          if (g < chains) sum += __uint_as_float(r[g][k]);
        v[k >> 3][k & 7] = sum;
      }
      if (C == 1) {
        finish(row, j / 8, v[0]);
        finish(row, j / 8 + 1, v[1]);
      } else if (row < rows8) {
        // [RP / 4][rows] of four ranks: a warp's 32 rows lie side by side
#pragma unroll
        for (int q = 0; q < 4; ++q)
          st_shared_f4(part + ((j / 4 + q) * rows8 + row) * 16u, v[q >> 1][4 * (q & 1)], v[q >> 1][4 * (q & 1) + 1],
                       v[q >> 1][4 * (q & 1) + 2], v[q >> 1][4 * (q & 1) + 3]);
      }
    }
    // -------------------------------------- the base's rows where they are copied
    // A warp copies its own 32 rows of its set's next tiles, `ahead` of them: nobody else reads them.
    int place[8];
#pragma unroll
    for (int p = 0; p < 8; ++p) place[p] = s_rows[quarter * 32 + 4 * p + sub];
    const int ahead = max(1, min(S2 - 1, early) / SETS);
    Turn fetch = {set, 0};
    int fetched = set;
    auto fetch_base = [&]() {
      if (fetched < tiles) {
        const int col = (nt0 + fetched) * kBk + 8 * ch;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const int r = quarter * 32 + 4 * p + sub;
          const bool there = place[p] >= 0 && col < N;
          if (r < t.nrows)
            copy16(sbase + fetch.slot * slot2 + swz(r, ch), base + (there ? static_cast<size_t>(place[p]) * N + col : 0),
                   there);
        }
      }
      copy_commit();
      fetched += SETS;
      fetch.step(SETS, S2);
    };
    const bool pre = early >= SETS * ahead;
    tc_fence_before();
    __syncwarp();
    cluster_arrive();
    if (copy_base && pre)
      for (int k = 0; k < ahead; ++k) fetch_base();
    __syncwarp();
    cluster_wait();
    if (C > 1) {
      // This CTA's rows of the tile, summed over the CTAs in their order.  Neighbouring lanes have
      // neighbouring rows, which lie in different banks of either tile.
      const int r0 = q_rows * rank / C, per = q_rows * (rank + 1) / C - r0;
      for (int i = tid - 64; i < per * (RP / 8); i += 128 * SETS) {
        const int r = r0 + i % per, j8 = i / per;
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        const uint32_t at = part + (2u * j8 * rows8 + r) * 16u;
        if (r < t.nrows) {
          constexpr int kAtOnce = SETS == 1 ? 4 : 8;  // CTAs: a load from another SM takes a while
          for (int p = 0; p < C; p += kAtOnce) {
            float4 x[2 * kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
              if (p + k >= C) break;
              const uint32_t from = map_to_cta(at, p + k);
              x[2 * k] = ld_cluster_f4(from);
              x[2 * k + 1] = ld_cluster_f4(from + rows8 * 16u);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
              if (p + k >= C) break;
              v[0] += x[2 * k].x, v[1] += x[2 * k].y, v[2] += x[2 * k].z, v[3] += x[2 * k].w;
              v[4] += x[2 * k + 1].x, v[5] += x[2 * k + 1].y, v[6] += x[2 * k + 1].z, v[7] += x[2 * k + 1].w;
            }
          }
        }
        finish(r, j8, v);
      }
    }
    fence_async_all();
    __syncwarp();
    cluster_sync();
    if (copy_base && !pre)
      for (int k = 0; k < ahead; ++k) fetch_base();
    // ------------------------------------------------------------ epilogue
    // A lane has a row: 64 columns of accumulators plus its base, in place in the slot.
    const bool by_tma = out_box && quarter * 32 + 32 <= t.nrows;
    const bool mine = row < rows8;
    int pend = -1;
    Turn to = {set, 0}, acc = {set, 0};
    for (int i = set; ok && i < tiles; i += SETS) {
      const uint32_t tile = sbase + to.slot * slot2;
      ok = wait_all(bar_bfull(to.slot), to.phase, abort_flag) && wait_all(bar_acc(acc.slot), acc.phase, abort_flag);
      if (!ok) break;
      tc_fence_after();
      if (copy_base) {
        copy_wait_left(ahead - 1);
        __syncwarp();
      }
      if (quarter * 32 < t.nrows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t r[32];
          tmem_ld_32x32b_x32(tq + acc.slot * kBk + 32 * h, r);
          uint4 b[4];
          if (base != nullptr && mine) {
#pragma unroll
            for (int c = 0; c < 4; ++c) b[c] = ld_shared_u4(tile + swz(row, 4 * h + c));
          }
          tmem_wait_ld();
          tmem_loaded(r);
          if (base != nullptr) {
            auto add2 = [](uint32_t u, uint32_t p, uint32_t q) {
              const float2 f = unpack_bf16(u);
              return pack_bf16(f.x + __uint_as_float(p), f.y + __uint_as_float(q));
            };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t* x = r + 8 * c;
              b[c].x = add2(b[c].x, x[0], x[1]);
              b[c].y = add2(b[c].y, x[2], x[3]);
              b[c].z = add2(b[c].z, x[4], x[5]);
              b[c].w = add2(b[c].w, x[6], x[7]);
            }
          } else {
            auto pack2 = [](uint32_t p, uint32_t q) { return pack_bf16(__uint_as_float(p), __uint_as_float(q)); };
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const uint32_t* x = r + 8 * c;
              b[c] = make_uint4(pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(x[4], x[5]), pack2(x[6], x[7]));
            }
          }
          if (mine) {
#pragma unroll
            for (int c = 0; c < 4; ++c) st_shared_u4(tile + swz(row, 4 * h + c), b[c]);
          }
        }
      }
      tc_fence_before();
      if (by_tma) fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_free(acc.slot));
      if (by_tma) {
        if (lane == 0) {
          if (pend >= 0) {
            bulk_wait_read0();  // this warp's tile before has left its slot
            mbar_arrive(bar_bempty(pend));
          }
          tma_store_2d(&a.tm_out, (nt0 + i) * kBk, t.row0 + quarter * 32, tile + quarter * 4096u);
          bulk_commit();
          pend = to.slot;
        }
      } else {
        const int col = (nt0 + i) * kBk + 8 * ch;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 v[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int q = quarter * 32 + 16 * h + 4 * p + sub;
            if (q < t.nrows) v[p] = ld_shared_u4(tile + swz(q, ch));
          }
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            const int o = place[4 * h + p];
            if (o >= 0 && col < N) *reinterpret_cast<uint4*>(out + static_cast<size_t>(o) * N + col) = v[p];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_bempty(to.slot));
      }
      if (copy_base) {
        // its slot has been read by the tile before in it, which may be the other set's
        if (fetched < tiles && fetched >= S2) ok = wait_all(bar_bempty(fetch.slot), fetch.phase ^ 1u, abort_flag);
        fetch_base();
      }
      to.step(SETS, S2);
      acc.step(SETS, kBufs);
    }
    if constexpr (TRANS) {
      // v's blocks, which the intermediate holds by rows
      if (a.qv != nullptr && ok) {
        for (int i = tid - 64; i < octets * RP * 2; i += 128 * SETS) {
          const int j = i % RP, part_of = i / RP & 1, o = rank + C * (i / (2 * RP));
          const uint32_t c = static_cast<uint32_t>(part_of * RQ + j);
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t r = 8u * o + 2 * k, at = su + (c >> 6) * kXBytes + 2u * (c & 7);
            const uint32_t x = ld_shared_u16(at + swz(r, (c & 63) >> 3));
            w[k] = x | ld_shared_u16(at + swz(r + 1, (c & 63) >> 3)) << 16;
          }
          *q_piece(a.qv, o, j, part_of) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    if (by_tma && lane == 0) bulk_wait_read0();
    copy_wait<0>();
    if (!ok && lane == 0) give_up(abort_flag, a.status);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <bool TRANS, int RQ, int SETS>
cudaError_t set_smem() {
  static thread_local uint64_t attr_ctx = 0;
  return set_smem_attr_once(reinterpret_cast<const void*>(lora_kernel<TRANS, RQ, SETS>), 227 * 1024, &attr_ctx);
}

cudaLaunchConfig_t config(int sets, int cluster, long long tiles, size_t smem, cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * cluster));
  cfg.blockDim = dim3(static_cast<unsigned>(threads_of(sets)));
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

constexpr int kMaxCluster = 8;
// Clusters of c CTAs, one to an SM, that the current context runs at once (none where it has a share of
// the SMs that is too small).  Asked once per context and thread.
template <bool TRANS, int RQ>
long long clusters_at_once(int c) {
  using P = Plan<RQ>;
  static thread_local uint64_t asked_ctx = 0;
  static thread_local int active[kMaxCluster + 1];
  if (asked_ctx == 0 || asked_ctx != current_context_id()) {
    for (int k = 2; k <= kMaxCluster; ++k) {
      cudaLaunchAttribute attr[2] = {};
      const cudaLaunchConfig_t cfg = config(kManySets, k, 1, P::smem(P::kLong), attr);
      if (cudaOccupancyMaxActiveClusters(&active[k], lora_kernel<TRANS, RQ, kManySets>, &cfg) != cudaSuccess) {
        (void)cudaGetLastError();  // a size that does not fit is no error of the call
        active[k] = 0;
      }
    }
    asked_ctx = current_context_id();
  }
  return active[c];
}

template <bool TRANS, int RQ, int SETS>
cudaError_t launch_sets(LoraArgs a, int cluster, long long tiles, cudaStream_t stream) {
  using P = Plan<RQ>;
  const cudaError_t err = set_smem<TRANS, RQ, SETS>();
  if (err != cudaSuccess) return err;
  a.cluster = cluster;
  a.ring = SETS == 1 ? P::kShort : P::kLong;
  cudaLaunchAttribute attr[2] = {};
  cudaLaunchConfig_t cfg = config(SETS, cluster, tiles, P::smem(a.ring), attr);
  cfg.stream = stream;
  return cudaLaunchKernelEx(&cfg, lora_kernel<TRANS, RQ, SETS>, a);
}

template <bool TRANS, int RQ>
cudaError_t launch(const LoraArgs& a, int num_sms, cudaStream_t stream) {
  cudaError_t err = set_smem<TRANS, RQ, kManySets>();
  if (err != cudaSuccess) return err;
  // The exact number of tiles is known on the device only: at most this many, one more for rows without
  // an adapter included; about half a tile of each adapter's is empty, or more where rows are few.
  const long long some = a.M < a.E ? a.M : a.E;
  const long long tiles = (a.M + kRows - 1) / kRows + some + 1;
  const long long full = (a.M + kRows - 1) / kRows, likely = full + some / 2 > some ? full + some / 2 : some;
  // Where the tiles leave SMs idle: as many CTAs to a tile, each with some columns of its own, as run at
  // once (a cluster that waits for another one's end costs as much again).
  const int nch = (a.K + kBk - 1) / kBk;
  const int most = a.max_cluster > 0 && a.max_cluster < kMaxCluster ? a.max_cluster : kMaxCluster;
  int c = 1;
  for (int k = 2; k <= most && k <= nch; ++k)
    if (likely <= clusters_at_once<TRANS, RQ>(k)) c = k;
  // More tiles than SMs: two CTAs to an SM, one's loads under the other's exchange.
  if constexpr (RQ < 128)
    if (likely > num_sms) return launch_sets<TRANS, RQ, 1>(a, 1, tiles, stream);
  return launch_sets<TRANS, RQ, kManySets>(a, c, tiles, stream);
}

template <bool TRANS>
cudaError_t launch_rank(const LoraArgs& a, int num_sms, cudaStream_t stream) {
  if (a.R > 64) return launch<TRANS, 128>(a, num_sms, stream);
  return a.R > 32 ? launch<TRANS, 64>(a, num_sms, stream) : launch<TRANS, 32>(a, num_sms, stream);
}

}  // namespace

cudaError_t launch_lora(const LoraArgs& a, bool transposed, int num_sms, cudaStream_t stream) {
  return transposed ? launch_rank<true>(a, num_sms, stream) : launch_rank<false>(a, num_sms, stream);
}

}  // namespace mgw
