// moe_int8_gemm.cu -- grouped products of the expert layer on 8-bit integers with
// one scale per row and per output column.
//
//   up:   h = bf16(silu(g) * u), g = sx swg (Qx Qwg^T), u = sx swu (Qx Qwu^T)
//   down: Y = bf16(sh swd (Qh Qwd^T))
// for the rows of each expert.  The integers reach the tensor cores as fp16, which
// holds them exactly (sm_103a has no integer MMA in tcgen05): their products are
// exact, and float32 sums of them stay exact while they are below 2^24.
//
// A tile is one window of up to 128 of an expert's rows times two blocks of 128
// output columns (up: the same columns of gate and of up; down: 256 neighbouring
// columns).  The weights are the M = 128 operand, the rows the N operand.  TMA
// brings the codes in stages of 128 k.  Two groups of eight warps widen them, each
// one half of every stage, a step of 64 k: the weights into TMEM, from where the
// MMA reads its first operand (lane = weight row, two k per column: a thread widens
// its own row), the rows into shared memory in the swizzle of the second operand.
// TMEM holds two 128 x 128 accumulators and kSteps such steps of both blocks.
//
// What bounds it with many rows is the widening: a step is 512 cycles of MMAs and
// about 440 of instruction issue, and a group needs some 800 from its wait to its
// arrival (one group alone: 1040 cycles a step, up product of 2048 tokens and 64
// experts of 4096 x 1536 444 us, of 16384 tokens and 128 experts 2914 us).
#include <cstdint>
#include <mutex>

#include <cuda_fp16.h>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_transpose.cuh"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kTok = 128;                 // most rows of a window
constexpr int kStageK = 128;              // reduction elements (bytes) per stage of codes
constexpr int kStepK = 64;                // and per widened step
constexpr int kStages = 3;
constexpr int kSteps = 4;
constexpr int kWBytes = 128 * kStageK;    // codes of one block of 128 weight rows
constexpr int kStageBytes = 2 * kWBytes + kTok * kStageK;
constexpr int kStepBytes = kTok * kStepK * 2;  // widened rows
// Warps: loads, MMAs, scheduler (and an idle one); epilogue; widening: whole groups
// of four warps, which share out the registers: kLaunchRegs a thread at launch,
// then what each group asks for.
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
constexpr int kReaders = 2 + kEpiWarps + kWideWarps;  // of a tile
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
constexpr int kSmem = kSlotOff + 16 + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

template <int kRegs>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs));
}
template <int kRegs>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs));
}

// D(tmem) (+)= A(tmem) B(smem), fp16 with float32 sums, 16 deep.
__device__ __forceinline__ void mma_f16_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 32 lanes x 32 columns: thread i's registers to lane i.
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
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
  uint64_t* full;   // [kTileRing] one arrival (the scheduler)
  uint64_t* empty;  // [kTileRing] kReaders arrivals
  int4* tile;       // [kTileRing]
};
__device__ __forceinline__ bool ring_put(const TileRing& r, uint32_t n, const Tile& c, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  if (!mbar_wait(&r.empty[slot], ((n / kTileRing) & 1u) ^ 1u, abort, status)) return false;
  volatile int* w = reinterpret_cast<volatile int*>(&r.tile[slot]);
  w[0] = c.rows | (c.alone ? 1 << 8 : 0) | (c.last ? 1 << 9 : 0);
  w[1] = c.e;
  w[2] = c.j;
  w[3] = c.row0;
  mbar_arrive(&r.full[slot]);
  return true;
}
// The n-th tile of this CTA, false when the wait gave up; the caller arrives on
// empty[n % kTileRing] afterwards.
__device__ __forceinline__ bool ring_get(const TileRing& r, uint32_t n, Tile& c, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  if (!mbar_wait(&r.full[slot], (n / kTileRing) & 1u, abort, status)) return false;
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

// Tiles are drawn from a counter in the workspace, in order: CTA b starts on tile
// b, and its scheduler warp (a lane knowing eight experts) draws every later
// index, finds the tile and hands it to the other roles.  Tile t: expert, column
// tile, window, so that the windows sharing a weight tile are neighbours; all of an
// expert's windows but the last have kTok rows.  The CTA that stops drawing last
// clears the counter, and knows whether the launch started from a cleared one:
// the word behind it counts the CTAs that have stopped (bits 0-9), sums their
// indexes plus one (bits 10-29), and gets bit 30 from the one that drew 0.  With
// anything else in either word the sum comes out wrong (tiles may have been left
// out): an error.
constexpr int kMaxGrid = 1023;
__device__ __forceinline__ uint32_t stopped(uint32_t ctas, uint32_t index_sum, bool drew_zero) {
  return ctas | (index_sum << 10) | (drew_zero ? 1u << 30 : 0u);
}
__device__ __forceinline__ void schedule(const TileRing& ring, int E, int NT, int64_t max_rows,
                                         const int32_t* off_pad, const int32_t* counts, int lane,
                                         volatile int* abort, uint32_t* status, uint32_t* sched) {
  constexpr int per = kMaxExperts / 32;
  const uint32_t all = 0xffffffffu;
  int cnt[per], off[per];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    cnt[i] = off[i] = 0;
    if (e < E) {
      const int c = __ldcg(counts + e);
      const int64_t first = __ldcg(off_pad + e), end = __ldcg(off_pad + e + 1);
      // an expert whose rows do not lie inside its 128-row blocks and the buffers
      // gets no tiles
      if (c >= 0 && first >= 0 && (first & 127) == 0 && (end & 127) == 0 && first + c <= end && end <= max_rows) {
        cnt[i] = c;
        off[i] = static_cast<int>(first);
      } else {
        record_status(status, kStatusBounds);
      }
    }
    sum += (cnt[i] + kTok - 1) / kTok;
  }
  int incl = sum;  // windows up to this lane's last expert
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(all, incl, o);
    if (lane >= o) incl += y;
  }
  const int windows = __shfl_sync(all, incl, 31);
  // windows of counts that fit the buffers (an expert has at most one that is not full)
  const bool fits = static_cast<int64_t>(windows - E) * kTok <= max_rows;
  if (!fits && lane == 0) record_status(status, kStatusBounds);
  const int total = fits ? NT * windows : 0;

  uint32_t drawn = 0, later = 0;  // two draws on their way
  if (lane == 0) {
    drawn = atomicAdd(sched, 1u);
    later = atomicAdd(sched, 1u);
  }
  bool drew_zero = false;
  int tile = blockIdx.x;
  for (uint32_t n = 0;; ++n) {
    Tile c{0, 0, 0, 0, false, tile >= total};
    int owner = 0;  // the lane that knows the tile's expert
    if (tile < total) {
      const int q = tile / NT;  // (all column tiles of a window's expert lie together)
      owner = __ffs(__ballot_sync(all, incl > q)) - 1;
      int base = incl - sum;  // windows before this lane's first expert
#pragma unroll
      for (int i = 0; i < per; ++i) {
        const int nw = (cnt[i] + kTok - 1) / kTok;
        if (q >= base && q < base + nw) {
          const int local = tile - NT * base;
          c.e = lane * per + i;
          c.j = local / nw;
          const int w = local - c.j * nw;
          c.row0 = off[i] + kTok * w;
          c.rows = min(kTok, cnt[i] - kTok * w);
          c.alone = nw == 1;
        }
        base += nw;
      }
    }
    bool put = true;
    if (lane == owner) put = ring_put(ring, n, c, abort, status);
    if (__any_sync(all, !put) || tile >= total) break;
    const uint32_t d = __shfl_sync(all, drawn, 0);
    drew_zero |= d == 0u;
    // a cleared counter gives less than total + 3 grids here
    const uint64_t next = static_cast<uint64_t>(gridDim.x) + d;
    if (next >= static_cast<uint64_t>(total) + 3u * gridDim.x && lane == 0) record_status(status, kStatusBounds);
    tile = next < static_cast<uint64_t>(total) ? static_cast<int>(next) : total;
    drawn = later;
    if (lane == 0) later = atomicAdd(sched, 1u);
  }
  if (lane == 0) {
    drew_zero |= drawn == 0u || later == 0u;
    __threadfence();
    const uint32_t mine = stopped(1u, blockIdx.x + 1u, drew_zero);
    const uint32_t seen = atomicAdd(sched + 1, mine) + mine;
    if ((seen & 0x3FFu) == gridDim.x) {  // every CTA has drawn its last index
      if (seen != stopped(gridDim.x, gridDim.x * (gridDim.x + 1u) / 2u, true)) record_status(status, kStatusBounds);
      atomicExch(sched, 0u);
      atomicExch(sched + 1, 0u);
    }
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

// silu(g) * u with the sigmoid on the SFU.  The exponent g log2 e is rounded
// before ex2, so below zero the relative error grows with |g|, to about
// |g| 2^-24 and a few ulps (2^-17 at g = -88, below which the result is the
// limit 0): far under h's rounding to bf16, 2^-9.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

template <bool kUp>
__global__ void __launch_bounds__(kThreads, 1)
    int8_gemm_kernel(const __grid_constant__ Int8Maps maps, const float* __restrict__ sT,
                     const float* __restrict__ sW0, const float* __restrict__ sW1, uint16_t* __restrict__ D,
                     const int32_t* __restrict__ off_pad, const int32_t* __restrict__ counts, int E, int K, int N_out,
                     int NT, int64_t max_rows, uint32_t* __restrict__ status, uint32_t* __restrict__ sched) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kBarOff);
  uint64_t* empty = full + kStages;
  uint64_t* wide = empty + kStages;   // a step is widened
  uint64_t* used = wide + kSteps;     // its MMAs are done
  uint64_t* tfull = used + kSteps;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tfull + 2;
  const TileRing ring{tfull + 3, tfull + 3 + kTileRing, reinterpret_cast<int4*>(smem + kRingOff)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kSlotOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kWideWarps);
    }
    for (int s = 0; s < kSteps; ++s) {
      mbar_init(&wide[s], kWideGroup);
      mbar_init(&used[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, kEpiWarps);
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
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
  const int KS = K / kStageK;

  if (warp < kFirstEpi) {
    fewer_registers<kControlRegs>();
    if (warp == 0) {
      // ---------------------------------------------------------- loads
      if (elect_one_sync()) {
        const uint64_t pol_keep = policy_evict_last();
        uint32_t it = 0;
        bool stop = false;
        Tile c;
        for (uint32_t n = 0; !stop && ring_get(ring, n, c, abort_flag, status) && !c.last; ++n) {
          mbar_arrive(&ring.empty[n % kTileRing]);
          // a one-window expert reads this weight tile once
          const uint64_t pol_w = c.alone ? policy_evict_first() : pol_keep;
          const int n0 = c.j * (kUp ? 128 : 256);
          const bool two = kUp || n0 + 128 < N_out;  // the second weight block exists
          const int w_row = c.e * N_out + n0;        // E * N_out < 2^31
          const int pick = c.rows <= 32 ? 0 : c.rows <= 64 ? 1 : 2;  // the smallest box that holds the window
          const uint32_t bytes = (two ? 2u : 1u) * kWBytes + int8_token_box(pick) * kStageK;
          for (int ks = 0; ks < KS; ++ks, ++it) {
            const uint32_t s = it % kStages;
            if (!mbar_wait(&empty[s], ((it / kStages) & 1u) ^ 1u, abort_flag, status)) {
              stop = true;
              break;
            }
            mbar_arrive_expect_tx(&full[s], bytes);
            uint8_t* st = smem + s * kStageBytes;
            const int kx = ks * kStageK;
            tma_load_2d(st, &maps.w0, &full[s], kx, w_row, pol_w);
            if (two)
              tma_load_2d(st + kWBytes, kUp ? &maps.w1 : &maps.w0, &full[s], kx, kUp ? w_row : w_row + 128, pol_w);
            tma_load_2d(st + 2 * kWBytes, &maps.t[pick], &full[s], kx, c.row0, pol_keep);
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
      // ---------------------------------------------------------- MMAs
      if (elect_one_sync()) {
        uint32_t it = 0;
        uint32_t tcount = 0;
        bool stop = false;
        Tile c;
        for (uint32_t n = 0; !stop && ring_get(ring, n, c, abort_flag, status) && !c.last; ++n) {
          mbar_arrive(&ring.empty[n % kTileRing]);
          const bool two = kUp || c.j * 256 + 128 < N_out;
          // fp16 operands, float32 sums, both with k contiguous, M = 128, N
          const uint32_t idesc = (1u << 4) | (static_cast<uint32_t>((c.rows + 15) / 16 * 2) << 17) | ((128u >> 4) << 24);
          if (!mbar_wait(tempty, (tcount & 1u) ^ 1u, abort_flag, status)) break;
          tc_fence_after();
          for (int ks = 0; ks < 2 * KS; ++ks, ++it) {
            const uint32_t s = it % kSteps;
            if (!mbar_wait(&wide[s], (it / kSteps) & 1u, abort_flag, status)) {
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
            tc_commit(&used[s]);
          }
          if (stop) break;
          tc_commit(tfull);
          ++tcount;
        }
        tc_commit(drain);
        int no_abort = 0;
        mbar_wait(drain, 0, &no_abort, status);
      }
      __syncwarp();
    } else if (warp == 2) {
      schedule(ring, E, NT, max_rows, off_pad, counts, lane, abort_flag, status, sched);
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
      bool ok = ring_get(ring, n, c, abort_flag, status);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[n % kTileRing]);
      const bool real = ok && !c.last;
      const int n0 = c.j * (kUp ? 128 : 256);
      const bool two = kUp || n0 + 128 < N_out;
      // the scales of this thread's columns 32 q + 8 x + lane / 4 of both blocks
      float w0[4], w1[4];
      if (real) {
        const int64_t at = static_cast<int64_t>(c.e) * N_out + n0 + 32 * q + (lane >> 2);
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          w0[x] = __ldcg(sW0 + at + 8 * x);
          w1[x] = two ? __ldcg((kUp ? sW1 : sW0 + 128) + at + 8 * x) : 0.0f;
        }
        ok = mbar_wait(tfull, tcount & 1u, abort_flag, status);
      }
      if (vote_any(!ok)) break;  // every warp gives up together (they share barriers)
      if (c.last) break;
      ++tcount;
      tc_fence_after();
      const int pieces = (c.rows + 31) / 32;
      const int mine = pieces > turn ? (pieces - turn + kTurns - 1) / kTurns : 0;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty);
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
          store(p, n0, pa[p]);
          if constexpr (!kUp) {
            if (two) store(p, n0 + 128, pb[p]);
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
    const int block = (w >> 2) & 1;   // weight block; of the rows, which half of a step's 16-byte chunks
    const int q = warp & 3;           // TMEM lane quarter; of the rows, which 32
    const int wrow = 32 * q + lane, trow = 32 * (w & 3) + lane;
    const uint32_t ta = tmem + (static_cast<uint32_t>(32 * q) << 16) + kWideCol + block * kWideBlockCols;
    uint32_t it = 0;
    bool stop = false;
    for (uint32_t n = 0; !stop; ++n) {
      Tile c{};
      const bool got = ring_get(ring, n, c, abort_flag, status);
      if (__any_sync(0xffffffffu, !got) || c.last) break;
      if (lane == 0) mbar_arrive(&ring.empty[n % kTileRing]);
      const bool two = kUp || c.j * 256 + 128 < N_out;
      const bool rows_here = 32 * (w & 3) < (c.rows + 15) / 16 * 16;
      for (int ks = 0; ks < KS && !stop; ++ks, ++it) {
        const uint32_t s = it % kStages;
        if (__any_sync(0xffffffffu, !mbar_wait(&full[s], (it / kStages) & 1u, abort_flag, status))) {
          stop = true;
          break;
        }
        const uint8_t* st = smem + s * kStageBytes;
        const uint32_t step = 2 * it + half, d = step % kSteps;
        if (__any_sync(0xffffffffu, !mbar_wait(&used[d], ((step / kSteps) & 1u) ^ 1u, abort_flag, status))) {
          stop = true;
          break;
        }
        tc_fence_after();
        if (block == 0 || two) {
          uint32_t r[32];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(st + block * kWBytes + swizzled(wrow, 4 * half + i));
            widen4(v.x, r[8 * i], r[8 * i + 1]);
            widen4(v.y, r[8 * i + 2], r[8 * i + 3]);
            widen4(v.z, r[8 * i + 4], r[8 * i + 5]);
            widen4(v.w, r[8 * i + 6], r[8 * i + 7]);
          }
          tmem_st_32x32b_x32(ta + d * 2 * kWideBlockCols, r);
        }
        if (rows_here) {
          uint8_t* to = smem + kStepOff + d * kStepBytes;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int ch = 2 * block + i;  // 16 k of the step
            const uint4 v = *reinterpret_cast<const uint4*>(st + 2 * kWBytes + swizzled(trow, 4 * half + ch));
            uint4 a, b;
            widen4(v.x, a.x, a.y);
            widen4(v.y, a.z, a.w);
            widen4(v.z, b.x, b.y);
            widen4(v.w, b.z, b.w);
            *reinterpret_cast<uint4*>(to + swizzled(trow, 2 * ch)) = a;
            *reinterpret_cast<uint4*>(to + swizzled(trow, 2 * ch + 1)) = b;
          }
          fence_proxy_async_smem();
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&wide[d]);
        if (lane == 0) mbar_arrive(&empty[s]);
      }
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
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
  const int NT = kUp ? N_out / 128 : (N_out + 255) / 256;
  const int64_t R = static_cast<int64_t>(s.T) * s.k;
  const int64_t max_tiles = (R / kTok + (s.E < R ? s.E : R)) * NT;
  if (num_sms > kMaxGrid) num_sms = kMaxGrid;
  const int grid = static_cast<int>(max_tiles < num_sms ? max_tiles : num_sms);
  return launch_pdl(int8_gemm_kernel<kUp>, dim3(grid), dim3(kThreads), kSmem, st, m, sT, sW0, sW1, D, off_pad, counts,
                    s.E, K, N_out, NT, max_rows_of(s), status, sched);
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
