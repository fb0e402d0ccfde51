// moe_int8_gemm.cu -- grouped products of the expert layer on 8-bit integers with
// one scale per row and per output column.
//
//   up:   h = bf16(silu(g) * u), g = sx swg (Qx Qwg^T), u = sx swu (Qx Qwu^T)
//   down: Y = bf16(sh swd (Qh Qwd^T))
// for the rows of each expert.  The integers reach the tensor cores as fp16, which
// holds them exactly (sm_103a has no integer MMA in tcgen05): their products are
// exact, and float32 sums of them stay exact while they are below 2^24.
//
// A cluster of two CTAs takes a tile: one window of up to 128 of an expert's rows
// times 256 output columns of gate and of up, or 512 of down.  The weights are the
// M = 256 operand (cta_group::2), two blocks of 128 rows in each CTA; the rows are
// the N operand, half of them supplied by either CTA.  TMA brings the codes in
// stages of 128 k.  In each CTA two groups of eight warps widen them, each one half
// of every stage, a step of 64 k: the weights into TMEM, from where the MMA reads
// its first operand (lane = weight row, two k per column: a thread widens its own
// row), the CTA's half of the rows into shared memory in the swizzle of the second
// operand.  TMEM holds two accumulators of 128 columns and kSteps such steps of
// both blocks.
//
// What bounds it with many rows is the MMAs and what of the widening they wait for:
// 2048 tokens and 64 experts of 4096 x 1536 take 292 us (gate/up; down 168), 16384
// tokens and 128 experts 1860 (1.77 PFLOP/s); with steps that are handed on unwidened
// the same tiles take 256 and 1617.  A group reads its codes before it waits for the
// step's buffers, so that shared memory's latency lies outside the chain from the MMA
// that frees a buffer to the one that reads it anew: 336, 192 and 2163 us with the
// reads behind the wait.  On single CTAs, which widen twice the rows and move 96 KB of
// shared memory a step instead of 64, 409, 212 and 2637 (reads behind the wait).  With
// 8 rows per expert 142 us, 5.7 TB/s of weights.
//
// Tried and slower, or no faster (reads behind the wait, 336 us, unless said): three
// groups in turn and four epilogue warps (367); four warps for the rows alone (391);
// the widened codes, not the codes, held across the wait (458: registers); a whole
// stage per group (345); one wait for both steps of a stage (354); one group (444, on
// single CTAs); with the reads ahead, the stage released right behind them (296, and
// 292 without).
#include <cstdint>
#include <mutex>

#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_epilogue.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kTok = 128;                 // most rows of a window
constexpr int kHalfTok = kTok / 2;        // of which a CTA supplies half
constexpr int kStageK = 128;              // reduction elements (bytes) per stage of codes
constexpr int kStepK = 64;                // and per widened step
constexpr int kStages = 4;
constexpr int kSteps = 4;
constexpr int kWBytes = 128 * kStageK;    // codes of one block of 128 weight rows
constexpr int kStageBytes = 2 * kWBytes + kHalfTok * kStageK;
constexpr int kStepBytes = kHalfTok * kStepK * 2;  // widened rows
// Warps: loads, MMAs and scheduler (both in CTA 0 alone) and an idle one; epilogue;
// widening: whole groups of four warps, which share out the registers: kLaunchRegs a
// thread at launch, then what each group asks for.
constexpr int kFirstEpi = 4;
constexpr int kEpiWarps = 8;
constexpr int kTurns = kEpiWarps / 4;
constexpr int kFirstWide = kFirstEpi + kEpiWarps;
constexpr int kWideGroup = 8;
constexpr int kWideWarps = 2 * kWideGroup;
constexpr int kThreads = (kFirstWide + kWideWarps) * 32;
constexpr int kLaunchRegs = 72, kControlRegs = 56, kEpiRegs = 112, kWideRegs = 56;
static_assert(kThreads * kLaunchRegs <= 65536 && kFirstEpi * kControlRegs + kEpiWarps * kEpiRegs +
                  kWideWarps * kWideRegs <= kThreads / 32 * kLaunchRegs, "registers");
constexpr int kTileRing = 4;                          // tiles on their way from the scheduler
constexpr int kReaders = 3 + 2 * (kEpiWarps + kWideWarps);  // of a tile, in both CTAs
// TMEM columns: the accumulators, then the widened weights of each step
constexpr uint32_t kAcc1 = kTok;
constexpr uint32_t kWideCol = 2 * kTok;
constexpr uint32_t kWideBlockCols = kStepK / 2;
static_assert(kWideCol + kSteps * 2 * kWideBlockCols <= 512, "TMEM columns");
constexpr int kStepOff = kStages * kStageBytes;
constexpr int kOutOff = kStepOff + kSteps * kStepBytes;
constexpr int kRingOff = kOutOff + kTurns * kPieceBytes;
constexpr int kBarOff = kRingOff + kTileRing * 16;
// full, empty [kStages]; wide, used [kSteps]; tfull, tempty, drain; the ring's
constexpr int kNumBars = 2 * kStages + 2 * kSteps + 3 + 2 * kTileRing;
constexpr int kSlotOff = kBarOff + kNumBars * 8;
constexpr int kRowsOff = kSlotOff + 16;              // the scheduler's counts and first rows
constexpr int kSmem = kRowsOff + kMaxExperts * 8 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// D(tmem) (+)= A(tmem) B(smem) over both CTAs, fp16 with float32 sums, 16 deep.
__device__ __forceinline__ void mma_f16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 16 columns: thread i's registers to lane i.
__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Four codes to two pairs of fp16: with its sign bit flipped a code is q + 128,
// which under the high byte 0x64 reads as 1024 + 128 + q.
__device__ __forceinline__ void widen4(uint32_t v, uint32_t& lo, uint32_t& hi) {
  const uint32_t b = v ^ 0x80808080u;
  const uint32_t magic = 0x64646464u;
  const __half2 bias = __half2half2(__ushort_as_half(0x6480));  // 1152
  uint32_t p = __byte_perm(b, magic, 0x4140), q = __byte_perm(b, magic, 0x4342);
  __half2 x = __hsub2(*reinterpret_cast<__half2*>(&p), bias), y = __hsub2(*reinterpret_cast<__half2*>(&q), bias);
  lo = *reinterpret_cast<uint32_t*>(&x);
  hi = *reinterpret_cast<uint32_t*>(&y);
}

// byte offset of row t, 16-byte chunk c (of 8) in rows of 128 bytes, 128-byte swizzle
__device__ __forceinline__ int swizzled(int t, int c) { return t * 128 + ((c ^ (t & 7)) << 4); }

// A tile as the scheduler hands it out.
struct Tile {
  int e, j, row0, rows;  // expert, column tile, first row and rows of the window
  bool alone;            // the expert has one window
  bool last;             // no tile: the roles end
};
struct TileRing {
  uint64_t* full;   // [kTileRing], this CTA: one arrival (the scheduler)
  uint64_t* empty;  // [kTileRing], used in CTA 0: kReaders arrivals
  int4* tile;       // [kTileRing], this CTA
};
__device__ __forceinline__ bool ring_put(const TileRing& r, uint32_t n, const Tile& c, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  if (!mbar_wait<true>(&r.empty[slot], ((n / kTileRing) & 1u) ^ 1u, abort, status)) return false;
  volatile int* w = reinterpret_cast<volatile int*>(&r.tile[slot]);
  const int x = c.rows | (c.alone ? 1 << 8 : 0) | (c.last ? 1 << 9 : 0);
  w[0] = x;
  w[1] = c.e;
  w[2] = c.j;
  w[3] = c.row0;
  mbar_arrive(&r.full[slot]);
  send_cluster(map_to_cta(&r.tile[slot], 1), map_to_cta(&r.full[slot], 1), make_int4(x, c.e, c.j, c.row0));
  return true;
}
// The n-th tile of this cluster, false when the wait gave up.
__device__ __forceinline__ bool ring_get(const TileRing& r, uint32_t n, uint32_t rank, Tile& c, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  const uint32_t ph = (n / kTileRing) & 1u;
  if (!(rank == 0 ? mbar_wait<false>(&r.full[slot], ph, abort, status)
                  : mbar_wait<true>(&r.full[slot], ph, abort, status)))
    return false;
  const volatile int* w = reinterpret_cast<const volatile int*>(&r.tile[slot]);
  const int x = w[0];
  c.rows = x & 255;
  c.alone = (x >> 8) & 1;
  c.last = (x >> 9) & 1;
  c.e = w[1];
  c.j = w[2];
  c.row0 = w[3];
  return true;
}

__device__ __forceinline__ void ring_release(const TileRing& r, uint32_t n, uint32_t rank, uint32_t empty0) {
  const uint32_t slot = n % kTileRing;
  if (rank == 0) mbar_arrive(&r.empty[slot]);
  else mbar_arrive_peer(empty0 + 8u * slot);
}

// Tiles are drawn from a counter in the workspace, in order: cluster b starts on
// tile b, and a warp of its CTA 0 (lane l knowing the experts l, 32 + l, ...) draws
// every later index, finds the tile and hands it to all roles of both CTAs (the first
// one before the first draws, whose latency the release to the readers would wait
// for).  Tile t: expert, column tile, window, so that the windows sharing a weight
// tile are neighbours; all of an expert's windows but the last have kTok rows.
__device__ __forceinline__ void schedule(const TileRing& ring, int E, int NT, int64_t max_rows,
                                         const int32_t* off_pad, const int32_t* counts, uint32_t cluster,
                                         uint32_t nclusters, int lane, volatile int* abort, uint32_t* status,
                                         uint32_t* sched, int2* known) {
  constexpr int kGroups = kMaxExperts / 32;  // of 32 experts
  const uint32_t all = 0xffffffffu;
  int cnt[kGroups], off[kGroups], end[kGroups];
  int incl[kGroups];  // windows up to the expert
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int e = 32 * i + lane;
    cnt[i] = off[i] = end[i] = 0;
    if (32 * i < E && e < E) {
      cnt[i] = __ldcg(counts + e);
      off[i] = __ldcg(off_pad + e);
      end[i] = __ldcg(off_pad + e + 1);
    }
  }
  int windows = 0;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    incl[i] = windows;
    if (32 * i < E) {
      // an expert whose rows do not lie inside its 128-row blocks and the buffers
      // gets no tiles
      if (cnt[i] < 0 || off[i] < 0 || (off[i] & 127) != 0 || (end[i] & 127) != 0 ||
          static_cast<int64_t>(off[i]) + cnt[i] > end[i] || end[i] > max_rows) {
        record_status(status, kStatusBounds);
        cnt[i] = 0;
      }
      known[32 * i + lane] = make_int2(cnt[i], off[i]);
      int sum = (cnt[i] + kTok - 1) / kTok;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(all, sum, o);
        if (lane >= o) sum += y;
      }
      incl[i] += sum;
      windows += __shfl_sync(all, sum, 31);
    }
  }
  // windows of counts that fit the buffers (an expert has at most one that is not full)
  const bool fits = static_cast<int64_t>(windows - E) * kTok <= max_rows;
  if (!fits && lane == 0) record_status(status, kStatusBounds);
  const int total = fits ? NT * windows : 0;

  uint32_t drawn = 0, later = 0;  // two draws on their way
  bool drew_zero = false;
  // every draw, of lane 0: a cleared counter gives less than total + 2 clusters
  auto checked = [&](uint32_t d) {
    drew_zero |= d == 0u;
    if (d >= static_cast<uint64_t>(total) + 2u * nclusters) record_status(status, kStatusBounds);
  };
  int tile = static_cast<int>(cluster);
  for (uint32_t n = 0;; ++n) {
    Tile c{0, 0, 0, 0, false, tile >= total};
    int owner = 0;  // the lane that knows the tile's expert
    if (tile < total) {
      const int q = tile / NT;  // (all column tiles of a window's expert lie together)
      int upto = 0;
      bool found = false;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        if (32 * i < E && !found) {
          const uint32_t behind = __ballot_sync(all, incl[i] > q);
          found = behind != 0u;
          if (found) {
            owner = __ffs(behind) - 1;
            c.e = 32 * i + lane;
            upto = incl[i];
          }
        }
      }
      const int2 mine = known[c.e];  // as this lane left it
      const int nw = (mine.x + kTok - 1) / kTok;
      const int local = tile - NT * (upto - nw);
      int w = 0;
      c.j = local;
      if (nw > 1) {
        c.j = local / nw;
        w = local - c.j * nw;
      }
      c.row0 = mine.y + kTok * w;
      c.rows = min(kTok, mine.x - kTok * w);
      c.alone = nw == 1;
    }
    bool put = true;
    if (lane == owner) put = ring_put(ring, n, c, abort, status);
    if (n == 0 && lane == 0) {
      drawn = atomicAdd(sched, 1u);
      later = atomicAdd(sched, 1u);
    }
    if (__any_sync(all, !put) || tile >= total) break;
    const uint32_t d = __shfl_sync(all, drawn, 0);
    if (lane == 0) checked(d);
    const uint64_t next = static_cast<uint64_t>(nclusters) + d;
    tile = next < static_cast<uint64_t>(total) ? static_cast<int>(next) : total;
    drawn = later;
    if (lane == 0) later = atomicAdd(sched, 1u);
  }
  if (lane == 0) {
    checked(drawn);
    checked(later);
    stop_drawing(sched, cluster, nclusters, drew_zero, true, status);
  }
}

// OR-vote over the epilogue's threads (named barrier 2).
__device__ __forceinline__ bool vote_any(bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 2, %2, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(flag ? 1u : 0u), "n"(kEpiWarps * 32)
      : "memory");
  return r != 0;
}

template <bool kUp>
__global__ void __launch_bounds__(kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ Int8Maps maps, const float* __restrict__ sT,
                     const float* __restrict__ sW0, const float* __restrict__ sW1, uint16_t* __restrict__ D,
                     const int32_t* __restrict__ off_pad, const int32_t* __restrict__ counts, int E, int K, int N_out,
                     int NT, int64_t max_rows, uint32_t* __restrict__ status, uint32_t* __restrict__ sched) {
  constexpr int kTileCols = kUp ? 256 : 512;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* empty = full + kStages;
  uint64_t* wide = empty + kStages;   // used in CTA 0: both CTAs have widened a step
  uint64_t* used = wide + kSteps;     // its MMAs are done
  uint64_t* tfull = used + kSteps;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tfull + 2;
  const TileRing ring{tfull + 3, tfull + 3 + kTileRing, reinterpret_cast<int4*>(smem + kRingOff)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: schedules and issues the MMAs
  // the first columns of the CTA's two blocks in a tile that starts at n0
  auto col_of = [&](int n0, int block) {
    return n0 + 128 * static_cast<int>(rank) + (kUp ? 0 : 256 * block);
  };

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWideWarps);
    }
    for (int s = 0; s < kSteps; ++s) {
      mbar_init(&wide[s], 2 * kWideGroup);
      mbar_init(&used[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, 2 * kEpiWarps);
    mbar_init(drain, 1);
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], kReaders);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&maps.t[0]);
    prefetch_tmap(&maps.w0);
    prefetch_tmap(&maps.w1);
    prefetch_tmap(&maps.out);
  }
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int KS = K / kStageK;
  const uint32_t wide0 = map_to_cta(wide, 0);
  const uint32_t tempty0 = map_to_cta(tempty, 0);
  const uint32_t rempty0 = map_to_cta(ring.empty, 0);

  if (warp < kFirstEpi) {
    fewer_registers<kControlRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- loads
      if (elect_one_sync()) {
        const uint64_t pol_keep = policy_evict_last();
        uint32_t it = 0;
        bool stop = false;
        Tile c;
        for (uint32_t n = 0; !stop && ring_get(ring, n, rank, c, abort_flag, status) && !c.last; ++n) {
          ring_release(ring, n, rank, rempty0);
          // a one-window expert reads this weight tile once
          const uint64_t pol_w = c.alone ? policy_evict_first() : pol_keep;
          const int c0 = col_of(c.j * kTileCols, 0), c1 = col_of(c.j * kTileCols, 1);
          const bool has0 = c0 < N_out, has1 = c1 < N_out;  // the blocks exist (columns are multiples of 128)
          const int w_row = c.e * N_out;                    // E * N_out < 2^31
          const int mine = (c.rows + 15) / 16 * 8;          // rows that this CTA supplies
          const int row = c.row0 + mine * static_cast<int>(rank);
          const int pick = mine <= 16 ? 0 : mine <= 32 ? 1 : 2;  // the smallest box that holds them
          const uint32_t bytes = (has0 ? kWBytes : 0) + (has1 ? kWBytes : 0) + int8_token_box(pick) * kStageK;
          for (int ks = 0; ks < KS; ++ks, ++it) {
            const uint32_t s = it % kStages;
            if (!mbar_wait(&empty[s], ((it / kStages) & 1u) ^ 1u, abort_flag, status)) {
              stop = true;
              break;
            }
            mbar_arrive_expect_tx(&full[s], bytes);
            uint8_t* st = smem + s * kStageBytes;
            const int kx = ks * kStageK;
            if (has0) tma_load_2d(st, &maps.w0, &full[s], kx, w_row + c0, pol_w);
            if (has1) tma_load_2d(st + kWBytes, kUp ? &maps.w1 : &maps.w0, &full[s], kx, w_row + c1, pol_w);
            tma_load_2d(st + 2 * kWBytes, &maps.t[pick], &full[s], kx, row, pol_keep);
          }
        }
        // every stage used must have been read before the CTA may exit
        const uint32_t nst = it < kStages ? it : kStages;
        for (uint32_t s = 0; s < nst; ++s) {
          const uint32_t last = s + kStages * ((it - 1 - s) / kStages);
          int no_abort = 0;
          mbar_wait(&empty[s], (last / kStages) & 1u, &no_abort, status);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ---------------------------------------------------------- MMAs (CTA 0)
      if (rank == 0 && elect_one_sync()) {
        uint32_t it = 0;
        uint32_t tcount = 0;
        bool stop = false;
        Tile c;
        for (uint32_t n = 0; !stop && ring_get(ring, n, rank, c, abort_flag, status) && !c.last; ++n) {
          ring_release(ring, n, rank, rempty0);
          const bool two = col_of(c.j * kTileCols, 1) < N_out;  // a second block in either CTA
          // fp16 operands, float32 sums, both with k contiguous, M = 256, N
          const uint32_t idesc =
              (1u << 4) | (static_cast<uint32_t>((c.rows + 15) / 16 * 2) << 17) | ((256u >> 4) << 24);
          if (!mbar_wait(tempty, (tcount & 1u) ^ 1u, abort_flag, status)) break;
          tc_fence_after();
          for (int ks = 0; ks < 2 * KS; ++ks, ++it) {
            const uint32_t s = it % kSteps;
            if (!mbar_wait<true>(&wide[s], (it / kSteps) & 1u, abort_flag, status)) {
              stop = true;
              break;
            }
            tc_fence_after();
            const uint32_t sb = smem_u32(smem + kStepOff + s * kStepBytes);
            const uint32_t ta = tmem + kWideCol + s * 2 * kWideBlockCols;
#pragma unroll
            for (int kk = 0; kk < kStepK / 16; ++kk) {
              const uint64_t bd = smem_desc(sb + kk * 32, 16, 1024, kSwizzle128B);
              const uint32_t acc = (ks | kk) != 0 ? 1u : 0u;
              mma_f16_tmem(tmem, ta + 8 * kk, bd, idesc, acc);
              if (two) mma_f16_tmem(tmem + kAcc1, ta + kWideBlockCols + 8 * kk, bd, idesc, acc);
            }
            tc_commit_pair(&used[s], 0x3);
          }
          if (stop) break;
          tc_commit_pair(tfull, 0x3);
          ++tcount;
        }
        tc_commit_pair(drain, 0x1);
        int no_abort = 0;
        mbar_wait(drain, 0, &no_abort, status);
      }
      __syncwarp();
    } else if (warp == 2 && rank == 0) {
      schedule(ring, E, NT, max_rows, off_pad, counts, blockIdx.x >> 1, gridDim.x >> 1, lane, abort_flag, status, sched,
               reinterpret_cast<int2*>(smem + kRowsOff));
      __syncwarp();
    }
  } else if (warp < kFirstWide) {
    more_registers<kEpiRegs>();
    // ---------------------------------------------------------- epilogue
    // TMEM lane = output column, TMEM column = row of the window; the warps of
    // a lane quarter take the window's 32-row pieces in turn
    const int q = warp & 3;
    const int turn = (warp - kFirstEpi) / 4;
    uint8_t* out = smem + kOutOff + turn * kPieceBytes;
    const uint32_t out_addr = smem_u32(out);
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const bool leader = q == 0 && lane == 0;
    uint32_t tcount = 0;
    for (uint32_t n = 0;; ++n) {
      Tile c{};
      bool ok = ring_get(ring, n, rank, c, abort_flag, status);
      const bool real = ok && !c.last;
      const int c0 = col_of(c.j * kTileCols, 0), c1 = col_of(c.j * kTileCols, 1);
      const bool has0 = c0 < N_out, two = c1 < N_out;
      // the scales of this thread's columns 32 q + 8 x + lane / 4 of both blocks
      float w0[4], w1[4];
      if (real) {
        const int64_t at = static_cast<int64_t>(c.e) * N_out + 32 * q + (lane >> 2);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          w0[x] = has0 ? __ldcg(sW0 + at + c0 + 8 * x) : 0.0f;
          w1[x] = two ? __ldcg((kUp ? sW1 : sW0) + at + c1 + 8 * x) : 0.0f;
        }
        ok = mbar_wait(tfull, tcount & 1u, abort_flag, status);
      }
      if (vote_any(!ok)) break;  // every warp gives up together (they share barriers)
      if (c.last) break;
      if (lane == 0) ring_release(ring, n, rank, rempty0);
      ++tcount;
      tc_fence_after();
      const int pieces = has0 ? (c.rows + 31) / 32 : 0;
      const int mine = pieces > turn ? (pieces - turn + kTurns - 1) / kTurns : 0;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(tempty0);
      };
      auto store = [&](int p, int col0, const uint32_t (&a)[16]) {
        const int64_t r0 = c.row0 + (turn + kTurns * p) * 32;
        const int left = c.rows - (turn + kTurns * p) * 32;
        if (leader) tma_store_wait_read<0>();
        __syncwarp();
        named_barrier_sync(3 + turn, 128);  // the previous piece has been read
        stage_piece(out_addr, q, a, lane);
        fence_proxy_async_smem();
        named_barrier_sync(3 + turn, 128);
        if (left >= 32) {  // alike for the turn's warps
          if (leader) {
            tma_store_2d(&maps.out, out, col0, static_cast<int32_t>(r0));
            tma_store_2d(&maps.out, out + kPieceBytes / 2, col0 + 64, static_cast<int32_t>(r0));
            tma_store_commit();
          }
          __syncwarp();
          return;
        }
        const int col = col0 + (lane & 15) * 8;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = 8 * q + 2 * i + (lane >> 4);
          if (t < left)
            *reinterpret_cast<uint4*>(D + (r0 + t) * N_out + col) =
                *reinterpret_cast<const uint4*>(out + staged_at(t, lane & 15));
        }
      };
      uint32_t pa[2][16], pb[kUp ? 1 : 2][16];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p < mine) {
          const int t0 = (turn + kTurns * p) * 32;
          float2 sx[4];  // of rows 8 j + 2 (lane % 4) and the next
#pragma unroll
          for (int j = 0; j < 4; ++j)
            sx[j] = __ldcg(reinterpret_cast<const float2*>(sT + c.row0 + t0 + 8 * j) + (lane & 3));
#pragma unroll
          for (int x2 = 0; x2 < 2; ++x2) {  // 16 TMEM lanes at a time
            uint32_t v0[16], v1[16];
            const uint32_t at = tb + (static_cast<uint32_t>(16 * x2) << 16) + t0;
            tmem_ld_16x256b_x4(at, v0);
            if (two) tmem_ld_16x256b_x4(at + kAcc1, v1);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {  // columns 8 (2 x2 + y) + lane / 4
                const int x = 2 * x2 + y, i = 4 * j + 2 * y;
                const float a0 = __uint_as_float(v0[i]) * sx[j].x * w0[x];
                const float a1 = __uint_as_float(v0[i + 1]) * sx[j].y * w0[x];
                const float b0 = __uint_as_float(v1[i]) * sx[j].x * w1[x];
                const float b1 = __uint_as_float(v1[i + 1]) * sx[j].y * w1[x];
                if constexpr (kUp) {
                  pa[p][4 * j + x] = pack_bf16x2(silu_mul(a0, b0), silu_mul(a1, b1));
                } else {
                  pa[p][4 * j + x] = pack_bf16x2(a0, a1);
                  pb[p][4 * j + x] = pack_bf16x2(b0, b1);
                }
              }
            }
          }
        }
      }
      release();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        if (p < mine) {
          store(p, c0, pa[p]);
          if constexpr (!kUp) {
            if (two) store(p, c1, pb[p]);
          }
        }
      }
    }
    if (leader) tma_store_wait_all<0>();  // this thread's stores are written
    __syncwarp();
  } else {
    fewer_registers<kWideRegs>();
    // ---------------------------------------------------------- widening
    const int w = warp - kFirstWide;
    const int half = w / kWideGroup;  // of each stage
    const int block = (w >> 2) & 1;   // weight block
    const int q = warp & 3;           // TMEM lane quarter
    const int wrow = 32 * q + lane;
    const int trow = 32 * (w & 1) + lane;  // of the rows: 32 of 64, and 16 k of the step
    const int ch = (w >> 1) & 3;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + kWideCol + block * kWideBlockCols;
    uint32_t it = 0;
    bool stop = false;
    for (uint32_t n = 0; !stop; ++n) {
      Tile c{};
      const bool got = ring_get(ring, n, rank, c, abort_flag, status);
      if (__any_sync(0xffffffffu, !got) || c.last) break;
      if (lane == 0) ring_release(ring, n, rank, rempty0);
      const bool block_here = col_of(c.j * kTileCols, block) < N_out;
      const bool rows_here = 32 * (w & 1) < (c.rows + 15) / 16 * 8;
      for (int ks = 0; ks < KS && !stop; ++ks, ++it) {
        const uint32_t s = it % kStages;
        if (__any_sync(0xffffffffu, !mbar_wait(&full[s], (it / kStages) & 1u, abort_flag, status))) {
          stop = true;
          break;
        }
        // the codes are read before the step's buffers are waited for
        const uint8_t* st = smem + s * kStageBytes;
        uint4 v[4], tv = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = *reinterpret_cast<const uint4*>(st + block * kWBytes + swizzled(wrow, 4 * half + i));
        if (rows_here) tv = *reinterpret_cast<const uint4*>(st + 2 * kWBytes + swizzled(trow, 4 * half + ch));
        const uint32_t step = 2 * it + half, d = step % kSteps;
        if (__any_sync(0xffffffffu, !mbar_wait(&used[d], ((step / kSteps) & 1u) ^ 1u, abort_flag, status))) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (block_here) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t r[16];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              widen4(v[2 * i + k].x, r[8 * k], r[8 * k + 1]);
              widen4(v[2 * i + k].y, r[8 * k + 2], r[8 * k + 3]);
              widen4(v[2 * i + k].z, r[8 * k + 4], r[8 * k + 5]);
              widen4(v[2 * i + k].w, r[8 * k + 6], r[8 * k + 7]);
            }
            tmem_st_32x32b_x16(ta + d * 2 * kWideBlockCols + 16 * i, r);
          }
        }
        if (rows_here) {
          uint8_t* to = smem + kStepOff + d * kStepBytes;
          uint4 a, b;
          widen4(tv.x, a.x, a.y);
          widen4(tv.y, a.z, a.w);
          widen4(tv.z, b.x, b.y);
          widen4(tv.w, b.z, b.w);
          *reinterpret_cast<uint4*>(to + swizzled(trow, 2 * ch)) = a;
          *reinterpret_cast<uint4*>(to + swizzled(trow, 2 * ch + 1)) = b;
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_peer(wide0 + 8u * d);
          mbar_arrive(&empty[s]);
        }
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  linger_after_abort(abort_flag);
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, 512);
  }
}

template <bool kUp>
cudaError_t launch(const moe_shape& s, const Int8Maps& m, const float* sT, const float* sW0, const float* sW1,
                   uint16_t* D, const int32_t* off_pad, const int32_t* counts, uint32_t* status, uint32_t* sched,
                   int num_sms, cudaStream_t st) {
  // the shared-memory opt-in, once per device (host threads may race here)
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      err = cudaFuncSetAttribute(int8_gemm_kernel<kUp>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (err != cudaSuccess) return err;
      if (dev < 64) done[dev] = true;
    }
  }
  const int K = kUp ? s.H : s.I;
  const int N_out = kUp ? s.I : s.H;
  constexpr int kCols = kUp ? 256 : 512;
  const int NT = (N_out + kCols - 1) / kCols;
  const int64_t R = static_cast<int64_t>(s.T) * s.k;
  const int64_t max_tiles = (R / kTok + (s.E < R ? s.E : R)) * NT;
  int64_t clusters = num_sms / 2;
  if (clusters > kMaxDrawers) clusters = kMaxDrawers;
  if (max_tiles < clusters) clusters = max_tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, int8_gemm_kernel<kUp>, m, sT, sW0, sW1, D, off_pad, counts, s.E, K, N_out, NT,
                            max_rows_of(s), status, sched);
}

}  // namespace

cudaError_t launch_int8_up(const moe_shape& s, const Int8Maps& m, const float* x_scales, const float* wg_scales,
                           const float* wu_scales, uint16_t* h, const int32_t* off_pad, const int32_t* counts,
                           uint32_t* status, uint32_t* sched, int num_sms, cudaStream_t st) {
  return launch<true>(s, m, x_scales, wg_scales, wu_scales, h, off_pad, counts, status, sched, num_sms, st);
}

cudaError_t launch_int8_down(const moe_shape& s, const Int8Maps& m, const float* h_scales, const float* wd_scales,
                             uint16_t* Y, const int32_t* off_pad, const int32_t* counts, uint32_t* status,
                             uint32_t* sched, int num_sms, cudaStream_t st) {
  return launch<false>(s, m, h_scales, wd_scales, wd_scales, Y, off_pad, counts, status, sched, num_sms, st);
}

}  // namespace moe
