// moe_mxfp4_gemm.cu -- grouped products of the expert layer on MXFP4 operands
// (block-scaled tcgen05.mma, kind::mxf4).
//
//   up:   h = bf16(silu(X Wg[e]) * (X Wu[e])), or that h quantised to MXFP4
//   down: Y = bf16(h Wd[e])
// for the rows of each expert e, both operands held as e2m1 codes with one
// e8m0 scale per 32 elements of the reduction axis; the tensor core applies
// the scales and accumulates in float32.
//
// A tile is one window of up to 128 or 192 (kTok) of an expert's rows times two
// blocks of 128 output columns (up: the same 128 columns of gate and of up;
// down: 256 neighbouring columns).  The weights are the M = 128 operand and the
// rows the N operand, so a window costs its row count rounded up to 16 and an
// output column's gate and up values meet in one thread.  TMEM holds the two
// 128 x N accumulators (lane = output column, column = row) and each stage's
// scales.  Windows start at multiples of kTok rows, so of 64: their rows' scales
// start at an even TMEM column of the 128-row scale tile.
//
// What bounds it: with 8 rows per expert (4096 x 1536, 64 experts, gate/up) the
// weights' bytes, 431 MB in 71 us = 6.1 TB/s (0.90 of the measured copy rate);
// with 1024 (128 experts) operand delivery: the tensor cores alone would take
// 458 us, the loads alone (8.5 GB from L2) 399 us, both together with the drain
// take 559 us, 5.9 PFLOP/s (608 us where a long run meets the power cap).
//
// The epilogue would cost as much as the MMAs if it held the accumulators, so
// its warps take them into registers (as raw sums as far as registers go,
// otherwise finished to bf16) and hand TMEM back; the rest of the arithmetic and
// all stores run under the next tile's MMAs.  (With the accumulators held to the
// end: 821 us where this takes 559.)
//
// Tried and slower: clusters of four sharing weights and rows by multicast (1352
// us: the CTAs wait for each other at every stage), of two sharing weights (738
// us), CTA pairs with cta_group::2 (573 us, down product 468 against 383), stages
// 128 deep (722 us).
//
// Roles of the warps: warp 0 loads (per 256-deep stage two boxes of 128 weight
// rows x 128 bytes, the window's rows in one box, and the scale tiles), warp 1
// copies a stage's scales to TMEM and issues its MMAs, the others drain the
// accumulators.  Every wait is bounded as in the bf16 GEMMs.
#include <cstdint>
#include <mutex>

#include "moe_epilogue.cuh"
#include "moe_internal.h"
#include "moe_mxfp4.cuh"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kStageK = 256;             // reduction elements per stage
constexpr int kAtoms = kStageK / 128;    // 128-deep scale tiles in a stage
constexpr int kRowBytes = kStageK / 2;   // codes of a row in a stage (128-byte swizzle)
constexpr int kWBytes = 128 * kRowBytes; // one block of 128 weight rows
constexpr int kSfBytes = 512 * kAtoms;   // scale tiles of 128 rows
constexpr int kFirstEpi = 2;             // epilogue warps follow the loading and the issuing one
constexpr int kTileRing = 4;             // tile indices on their way from the producer

// What depends on the most rows of a window.
template <int kTok>
struct Cfg {
  static_assert(kTok == 128 || kTok == 192, "windows start at an even column of their scale tile");
  // 64 columns of each accumulator per epilogue warp, in pieces of 32
  static constexpr int EPI_WARPS = kTok / 16;
  static constexpr int EPI_SPLIT = EPI_WARPS / 4;          // warps sharing a lane quarter
  static constexpr int PIECES = kTok / 32 / EPI_SPLIT;
  static_assert(PIECES == 2, "the epilogue's shape");
  static constexpr int THREADS = (kFirstEpi + EPI_WARPS) * 32;
  static constexpr int READERS = 1 + EPI_WARPS;  // of a tile index: the MMA lane, a lane of each epilogue warp
  // Pieces that a warp may keep as raw sums until TMEM is free: 64 registers
  // each, of 168 with ten warps, of 128 with fourteen.
  static constexpr int RAW = kTok == 128 ? 2 : 1;
  static constexpr int STAGES = kTok == 128 ? 4 : 3;
  static constexpr int SF_BLOCKS = kTok == 128 ? 1 : 2;    // 128-row scale blocks that a window's rows reach
  static constexpr int OFF_T = 2 * kWBytes;
  static constexpr int OFF_SF = OFF_T + kTok * kRowBytes;  // scales: weights 0, weights 1, rows
  static constexpr int STAGE_BYTES = OFF_SF + (2 + SF_BLOCKS) * kSfBytes;
  // TMEM columns: the accumulators, then each stage's scales (per 128 k:
  // weights 0 +0, weights 1 +4, rows +8)
  static constexpr uint32_t ACC1 = kTok;
  static constexpr uint32_t SF_COL = 2 * kTok;
  static constexpr uint32_t SF_STAGE_COLS = 16 * kAtoms;
  static constexpr int BAR_OFF = STAGES * STAGE_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 3 + 2 * kTileRing;
  static constexpr int TILE_OFF = BAR_OFF + NUM_BARS * 8 + 8;
  static constexpr int WIN_OFF = TILE_OFF + kTileRing * 4;
  static constexpr int CNT_OFF = WIN_OFF + (kMaxExperts + 1) * 4;
  static constexpr int OFFP_OFF = CNT_OFF + kMaxExperts * 4;
  static constexpr int OUT_OFF = (OFFP_OFF + (kMaxExperts + 1) * 4 + 1023) / 1024 * 1024;
  static constexpr int ALLOC = OUT_OFF + EPI_SPLIT * kPieceBytes + 1024;
  static_assert(STAGE_BYTES % 1024 == 0, "stages start on swizzle atoms");
  static_assert(SF_COL + STAGES * SF_STAGE_COLS <= 512, "TMEM columns");
  static_assert(ALLOC <= 232448, "shared memory budget");
};

enum Mode { kUpBf16 = 0, kUpMxfp4 = 1, kDown = 2 };

// Untiled copy of `bytes` (a multiple of 16, both sides 16-byte aligned)
// global -> shared, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// One 512-byte scale tile (128 rows x 4 blocks) from shared memory into four
// TMEM columns, replicated to the four 32-lane quarters: lane i, column c
// holds the scale word of row 32 c + i.
__device__ __forceinline__ void sf_to_tmem(uint32_t tmem, uint32_t smem) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(tmem), "l"(smem_desc(smem, 0, 128, 0))
               : "memory");
}

// D(tmem) (+)= A(smem) B(smem), both e2m1 with e8m0 scales per 32 elements,
// 64 elements deep.
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
      : "memory");
}

// kind::mxf4 instruction descriptor: A and B e2m1 (bits 7-9 and 10-11 = 1),
// both K-major, N >> 3 in bits 17-22, scales e8m0 (bit 23), M >> 7 in bits
// 27-28; `half` picks which two scales of each word a 64-deep step uses (byte
// 0 or 2, bits 4-5 for B and 29-30 for A).
__device__ __forceinline__ uint32_t idesc_mxf4(uint32_t N, uint32_t half) {
  return (1u << 7) | (1u << 10) | ((N >> 3) << 17) | (1u << 23) | (1u << 27) | ((2u * half) << 4) |
         ((2u * half) << 29);
}

struct Win {
  int e, j, row0, rows;
  bool ok;
};

// Tile t: expert e (windows off[e] .. off[e+1]), then column tile j, then the
// window, so that the windows sharing a weight tile are neighbours.  All of an
// expert's windows but the last have kTok rows.
template <int kTok>
__device__ __forceinline__ Win decode(int tile, int NT, int E, const int32_t* off, const int32_t* offp,
                                      const int32_t* cnt, int64_t max_rows) {
  Win c{0, 0, 0, 0, false};
  const int q = tile / NT;
  int lo = 0, hi = E;  // last e with off[e] <= q
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (off[mid] <= q) lo = mid; else hi = mid - 1;
  }
  if (lo >= E) return c;
  const int nw = off[lo + 1] - off[lo];
  const int local = tile - NT * off[lo];
  if (nw <= 0 || local < 0 || local >= NT * nw) return c;
  const int w = local % nw;
  c.e = lo;
  c.j = local / nw;
  // the window's rows lie inside the expert's 128-row blocks, and those inside
  // the buffers, whatever the counts and offsets given
  const int64_t first = offp[lo], row0 = first + static_cast<int64_t>(kTok) * w, pad_end = offp[lo + 1];
  c.rows = min(kTok, cnt[lo] - kTok * w);
  c.ok = c.rows > 0 && first >= 0 && (first & 127) == 0 && (pad_end & 127) == 0 && row0 + c.rows <= pad_end &&
         pad_end <= max_rows;
  c.row0 = static_cast<int>(row0);
  return c;
}

// Tiles are drawn from a counter in the workspace, in order (CTA b starts on
// tile b): windows differ in rows, and CTAs that got short ones take more.  The
// producer publishes each index to the other roles through a ring in shared
// memory; the CTA that stops drawing last clears the counter for the next
// launch and checks that it was clear.
struct TileRing {
  uint64_t* full;         // [kTileRing] one arrival (the producer)
  uint64_t* empty;        // [kTileRing] Cfg::READERS arrivals
  volatile int32_t* idx;  // [kTileRing]
};
__device__ __forceinline__ bool ring_put(const TileRing& r, uint32_t n, int tile, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  if (!mbar_wait(&r.empty[slot], ((n / kTileRing) & 1u) ^ 1u, abort, status)) return false;
  r.idx[slot] = tile;
  mbar_arrive(&r.full[slot]);
  return true;
}

// The n-th tile of this CTA, -1 when the wait gave up; the caller arrives on
// empty[n % kTileRing] afterwards.
__device__ __forceinline__ int ring_take(const TileRing& r, uint32_t n, volatile int* abort, uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  return mbar_wait(&r.full[slot], (n / kTileRing) & 1u, abort, status) ? r.idx[slot] : -1;
}

// One warp: the windows of up to kTok rows that each expert's count makes, their
// exclusive scan to win[0..E], and the counts to cnt (E <= 256).
template <int kTok>
__device__ __forceinline__ void scan_windows(const int32_t* counts, int E, int64_t max_rows, int32_t* win,
                                             int32_t* cnt, int lane, uint32_t* status) {
  constexpr int per = kMaxExperts / 32;
  int loc[per];
  int sum = 0;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    int nw = 0;
    if (e < E) {
      int c = __ldcg(counts + e);
      if (c > max_rows) {  // no buffer holds so many: no tiles for them
        record_status(status, kStatusBounds);
        c = 0;
      }
      cnt[e] = c;
      nw = c > 0 ? (c - 1) / kTok + 1 : 0;
    }
    loc[i] = nw;
    sum += nw;
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  int run = incl - sum;
#pragma unroll
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e <= E) win[e] = run;
    run += loc[i];
  }
  if (lane == 31 && 32 * per == E) win[E] = incl;
}

// OR-vote over the epilogue's threads (named barrier 2).
template <int kCount>
__device__ __forceinline__ bool vote_any(bool flag) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, 2, %2, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(flag ? 1u : 0u), "n"(kCount)
      : "memory");
  return r != 0;
}

// The same of silu(g) * u.
__device__ __forceinline__ void gate_piece(const uint32_t (&g)[32], const uint32_t (&u)[32], uint32_t (&out)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const int i = piece_entry(k);
    out[k] = pack_bf16x2(silu_mul(__uint_as_float(g[i]), __uint_as_float(u[i])),
                         silu_mul(__uint_as_float(g[i + 1]), __uint_as_float(u[i + 1])));
  }
}

template <int kMode, int kTok>
__global__ void __launch_bounds__(Cfg<kTok>::THREADS, 1)
    mxfp4_gemm_kernel(const __grid_constant__ Mxfp4Maps maps, const uint8_t* __restrict__ sfT,
                      const uint8_t* __restrict__ sfW0, const uint8_t* __restrict__ sfW1, void* __restrict__ D,
                      uint8_t* __restrict__ Dsf, const int32_t* __restrict__ off_pad,
                      const int32_t* __restrict__ counts, int E, int K, int N_out, int NT, int64_t max_rows,
                      uint32_t* __restrict__ status, uint32_t* __restrict__ sched) {
  using C = Cfg<kTok>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tfull = empty + C::STAGES;
  uint64_t* tempty = tfull + 1;
  uint64_t* drain = tfull + 2;
  const TileRing ring{tfull + 3, tfull + 3 + kTileRing, reinterpret_cast<volatile int32_t*>(smem + C::TILE_OFF)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tfull + 3 + 2 * kTileRing);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* s_win = reinterpret_cast<int32_t*>(smem + C::WIN_OFF);
  int32_t* s_cnt = reinterpret_cast<int32_t*>(smem + C::CNT_OFF);
  int32_t* s_offp = reinterpret_cast<int32_t*>(smem + C::OFFP_OFF);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
    mbar_init(tempty, C::EPI_WARPS);
    mbar_init(drain, 1);
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], C::READERS);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&maps.t[0]);
    prefetch_tmap(&maps.w0);
    prefetch_tmap(&maps.w1);
    if (kMode != kUpMxfp4) prefetch_tmap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  pdl_wait();
  if (warp == 2) {
    scan_windows<kTok>(counts, E, max_rows, s_win, s_cnt, lane, status);
  } else if (warp == 3) {
    for (int e = lane; e <= E; e += 32) s_offp[e] = __ldcg(off_pad + e);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // windows of counts that fit the buffers: the full ones hold kTok of max_rows
  // rows each, and an expert has one more at most (so total < 2^28).  Counts that
  // ask for more give no tiles.
  const bool fits = static_cast<int64_t>(s_win[E] - E) * kTok <= max_rows;
  if (!fits && threadIdx.x == 0) record_status(status, kStatusBounds);
  const int total = fits ? NT * s_win[E] : 0;
  const int KT = K / 128;  // scale tiles along the reduction
  const int KS = (KT + kAtoms - 1) / kAtoms;

  if (warp == 0) {
    // ---------------------------------------------------------- loads
    if (elect_one_sync()) {
      const uint64_t pol_t = policy_evict_last();
      uint32_t it = 0;
      int tile = blockIdx.x;
      bool drew_zero = false;
      bool stop = !ring_put(ring, 0, tile, abort_flag, status);
      for (uint32_t n = 0; !stop && tile < total; ++n) {
        const uint32_t drawn = atomicAdd(sched, 1u);  // the next tile: needed after this one's loads
        const Win c = decode<kTok>(tile, NT, E, s_win, s_offp, s_cnt, max_rows);
        if (!c.ok) record_status(status, kStatusBounds);
        // a one-window expert reads this weight tile once; otherwise its windows
        // share it, and it outlasts the output (gate/up of 16384 tokens 1.5%
        // faster than with the normal priority)
        const uint64_t pol_w = s_win[c.e + 1] - s_win[c.e] == 1 ? policy_evict_first() : pol_t;
        const int n0 = c.j * (kMode == kDown ? 256 : 128);
        const bool two = kMode != kDown || n0 + 128 < N_out;  // the second weight block exists
        const int w_row = c.e * N_out + n0;                   // E * N_out < 2^31
        // the smallest box that holds the window (rows past it are not used)
        const int pick = c.rows <= 32 ? 0 : c.rows <= 64 ? 1 : c.rows <= 128 ? 2 : 3;
        const int box = mxfp4_token_box(pick);
        const bool t_two = C::SF_BLOCKS > 1 && (c.row0 & 127) + c.rows > 128;  // its rows span two scale blocks
        for (int ks = 0; c.ok && ks < KS; ++ks, ++it) {
          const uint32_t s = it % C::STAGES;
          if (!mbar_wait(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, status)) {
            stop = true;
            break;
          }
          const int kt = min(kAtoms, KT - kAtoms * ks);  // scale tiles in this stage
          const uint32_t sfb = 512u * kt;
          mbar_arrive_expect_tx(&full[s],
                                (two ? 2u : 1u) * (kWBytes + sfb) + box * kRowBytes + (t_two ? 2u : 1u) * sfb);
          uint8_t* st = smem + s * C::STAGE_BYTES;
          const int kx = ks * kRowBytes;
          tma_load_2d(st, &maps.w0, &full[s], kx, w_row, pol_w);
          if (two)
            tma_load_2d(st + kWBytes, kMode == kDown ? &maps.w0 : &maps.w1, &full[s], kx,
                        kMode == kDown ? w_row + 128 : w_row, pol_w);
          tma_load_2d(st + C::OFF_T, &maps.t[pick], &full[s], kx, c.row0, pol_t);
          uint8_t* sf = st + C::OFF_SF;
          const int64_t wsf = (static_cast<int64_t>(w_row >> 7) * KT + kAtoms * ks) * 512;
          const int64_t tsf = (static_cast<int64_t>(c.row0 >> 7) * KT + kAtoms * ks) * 512;
          bulk_load(sf, sfW0 + wsf, sfb, &full[s]);
          if (two) bulk_load(sf + kSfBytes, kMode == kDown ? sfW0 + wsf + KT * 512 : sfW1 + wsf, sfb, &full[s]);
          bulk_load(sf + 2 * kSfBytes, sfT + tsf, sfb, &full[s]);
          if (t_two) bulk_load(sf + 3 * kSfBytes, sfT + tsf + KT * 512, sfb, &full[s]);
        }
        drew_zero |= drawn == 0u;
        if (stop) break;
        // a cleared counter gives at most total + grid - 1 here
        const uint64_t next = static_cast<uint64_t>(gridDim.x) + drawn;
        tile = next < static_cast<uint64_t>(total) + gridDim.x ? static_cast<int>(next) : total;
        if (static_cast<uint64_t>(tile) != next) record_status(status, kStatusBounds);
        stop = !ring_put(ring, n + 1, tile, abort_flag, status);
      }
      stop_drawing(sched, blockIdx.x, gridDim.x, drew_zero, total > 0, status);
      // every stage used must be consumed before the CTA may exit
      const uint32_t nst = it < C::STAGES ? it : C::STAGES;
      for (uint32_t s = 0; s < nst; ++s) {
        const uint32_t last = s + C::STAGES * ((it - 1 - s) / C::STAGES);
        int no_abort = 0;
        mbar_wait(&empty[s], (last / C::STAGES) & 1u, &no_abort, status);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMAs
    if (elect_one_sync()) {
      uint32_t it = 0;
      uint32_t tcount = 0;
      bool stop = false;
      for (uint32_t n = 0; !stop; ++n) {
        const int tile = ring_take(ring, n, abort_flag, status);
        if (tile < 0 || tile >= total) break;
        mbar_arrive(&ring.empty[n % kTileRing]);
        const Win c = decode<kTok>(tile, NT, E, s_win, s_offp, s_cnt, max_rows);
        if (!c.ok) continue;
        const bool two = kMode != kDown || c.j * 256 + 128 < N_out;
        const uint32_t N = static_cast<uint32_t>((c.rows + 15) / 16 * 16);
        const uint32_t id[2] = {idesc_mxf4(N, 0), idesc_mxf4(N, 1)};
        const bool t_two = C::SF_BLOCKS > 1 && (c.row0 & 127) + c.rows > 128;
        const uint32_t t_col = (c.row0 & 127) / 32;  // first row's column inside its scale block: 0 or 2
        if (!mbar_wait(tempty, (tcount & 1u) ^ 1u, abort_flag, status)) break;
        tc_fence_after();
        for (int ks = 0; ks < KS; ++ks, ++it) {
          const uint32_t s = it % C::STAGES;
          if (!mbar_wait(&full[s], (it / C::STAGES) & 1u, abort_flag, status)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_u32(smem + s * C::STAGE_BYTES);
          const uint32_t sf = st + C::OFF_SF;
          const uint32_t tsf = tmem + C::SF_COL + s * C::SF_STAGE_COLS;  // this stage's own columns
          const int kt = min(kAtoms, KT - kAtoms * ks);
          for (int a = 0; a < kt; ++a) {
            sf_to_tmem(tsf + 16 * a, sf + 512 * a);
            if (two) sf_to_tmem(tsf + 16 * a + 4, sf + kSfBytes + 512 * a);
            sf_to_tmem(tsf + 16 * a + 8, sf + 2 * kSfBytes + 512 * a);
            if (t_two) sf_to_tmem(tsf + 16 * a + 12, sf + 3 * kSfBytes + 512 * a);
          }
          for (int kk = 0; kk < 2 * kt; ++kk) {  // 64 deep each
            const uint64_t bd = smem_desc(st + C::OFF_T + kk * 32, 16, 8 * kRowBytes, kSwizzle128B);
            const uint32_t sfc = tsf + 16 * (kk >> 1);
            const uint32_t acc = (ks | kk) != 0 ? 1u : 0u;
            mma_mxf4(tmem, smem_desc(st + kk * 32, 16, 8 * kRowBytes, kSwizzle128B), bd, id[kk & 1], sfc,
                     sfc + 8 + t_col, acc);
            if (two)
              mma_mxf4(tmem + C::ACC1, smem_desc(st + kWBytes + kk * 32, 16, 8 * kRowBytes, kSwizzle128B), bd,
                       id[kk & 1], sfc + 4, sfc + 8 + t_col, acc);
          }
          tc_commit(&empty[s]);
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
  } else {
    // ---------------------------------------------------------- epilogue
    // TMEM lane = output column, TMEM column = row of the window; the warps of
    // a lane quarter take the window's 32-row pieces in turn
    const int q = warp & 3;
    const int turn = (warp - kFirstEpi) / 4;
    uint8_t* out = smem + C::OUT_OFF + turn * kPieceBytes;
    const uint32_t out_addr = smem_u32(out);
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t tcount = 0;
    for (uint32_t n = 0;; ++n) {
      const int tile = ring_take(ring, n, abort_flag, status);
      __syncwarp();
      if (lane == 0) mbar_arrive(&ring.empty[n % kTileRing]);
      bool ok = tile >= 0;
      const Win c = decode<kTok>(ok && tile < total ? tile : 0, NT, E, s_win, s_offp, s_cnt, max_rows);
      if (ok && tile < total && c.ok) ok = mbar_wait(tfull, tcount & 1u, abort_flag, status);
      if (vote_any<C::EPI_WARPS * 32>(!ok)) break;  // every warp gives up together (they share barriers)
      if (tile >= total) break;
      if (!c.ok) continue;
      ++tcount;
      tc_fence_after();
      const int n0 = c.j * (kMode == kDown ? 256 : 128);
      const bool two = kMode != kDown || n0 + 128 < N_out;
      const int pieces = (c.rows + 31) / 32;
      const int mine = pieces > turn ? (pieces - turn + C::EPI_SPLIT - 1) / C::EPI_SPLIT : 0;
      auto fetch = [&](int p, uint32_t (&v0)[32], uint32_t (&v1)[32]) {
        load_piece(tb + (turn + C::EPI_SPLIT * p) * 32, v0);
        if (two) load_piece(tb + C::ACC1 + (turn + C::EPI_SPLIT * p) * 32, v1);
      };
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(tempty);
      };
      // A finished piece of the 128 output columns from `col0` to the window's
      // rows: the turn's four warps put it together in shared memory; 32 rows of
      // bf16 then leave by TMA (written by the warps they held up the epilogue:
      // down product of 16384 tokens 388 us, this way 367), fewer rows and
      // quantised ones are written by the warps, eight rows each, sixteen lanes a
      // row.
      auto store = [&](int p, int col0, const uint32_t (&a)[16]) {
        const int64_t r0 = c.row0 + (turn + C::EPI_SPLIT * p) * 32;
        const int left = c.rows - (turn + C::EPI_SPLIT * p) * 32;
        if (kMode != kUpMxfp4 && q == 0) {
          if (lane == 0) tma_store_wait_read<0>();
          __syncwarp();
        }
        named_barrier_sync(3 + turn, 128);  // the previous piece has been read
        stage_piece(out_addr, q, a, lane);
        if (kMode != kUpMxfp4) fence_proxy_async_smem();
        named_barrier_sync(3 + turn, 128);
        if (kMode != kUpMxfp4 && left >= 32) {  // alike for the turn's warps
          if (q == 0 && lane == 0) {
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
          const uint4 h = *reinterpret_cast<const uint4*>(out + staged_at(t, lane & 15));
          if constexpr (kMode == kUpMxfp4) {
            // four lanes hold a block: the codes are those of quantising the
            // bf16 h
            const uint32_t s = block_scale_of_quad(h);
            const uint32_t w = scale_word_of_half(s, lane);
            if (t < left) {
              *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(D) + ((r0 + t) * N_out + col) / 2) =
                  quantize_bf16x8(h, s);
              if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t*>(Dsf + scale_word_offset(r0 + t, col0 / 128, N_out / 128)) = w;
            }
          } else {
            if (t < left) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(D) + (r0 + t) * N_out + col) = h;
          }
        }
      };
      auto store_all = [&](int p, const uint32_t (&a)[16], const uint32_t (&b)[16]) {
        store(p, n0, a);
        if constexpr (kMode == kDown) {
          if (two) store(p, n0 + 128, b);
        }
      };
      uint32_t va[C::RAW][32], vb[C::RAW][32], done[16];  // raw pieces, a finished one
      if constexpr (kMode == kDown) {
        // rounding is all there is to do: every piece is finished as it is read
        // (keeping raw sums, with windows of 128: 97 us for 73, T 2048)
        uint32_t pa[2][16], pb[2][16];
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (p < mine) {
            load_piece(tb + (turn + C::EPI_SPLIT * p) * 32, va[0]);
            tmem_ld_wait();
            round_piece(va[0], pa[p]);
            if (two) {
              load_piece(tb + C::ACC1 + (turn + C::EPI_SPLIT * p) * 32, va[0]);
              tmem_ld_wait();
              round_piece(va[0], pb[p]);
            }
          }
        }
        release();
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if (p < mine) store_all(p, pa[p], pb[p]);
      } else if constexpr (C::RAW == 2) {
        // every piece is kept as it is until TMEM is free
#pragma unroll
        for (int p = 0; p < 2; ++p)
          if (p < mine) fetch(p, va[p], vb[p]);
        tmem_ld_wait();
        release();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          if (p < mine) {
            gate_piece(va[p], vb[p], done);
            store(p, n0, done);
          }
        }
      } else if (mine == 0) {
        release();
      } else {
        // the first of two pieces is finished, the last kept as it is
        fetch(0, va[0], vb[0]);
        tmem_ld_wait();
        if (mine == 2) {
          gate_piece(va[0], vb[0], done);
          fetch(1, va[0], vb[0]);
          tmem_ld_wait();
        }
        release();
        if (mine == 2) store(0, n0, done);
        gate_piece(va[0], vb[0], done);
        store(mine - 1, n0, done);
      }
    }
    if (kMode != kUpMxfp4 && q == 0 && lane == 0) tma_store_wait_all<0>();  // this thread's stores are written
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

template <int kMode, int kTok>
cudaError_t launch_tok(const moe_shape& s, const Mxfp4Maps& m, const uint8_t* sfT, const uint8_t* sfW0,
                   const uint8_t* sfW1, void* D, uint8_t* Dsf, const int32_t* off_pad, const int32_t* counts,
                   uint32_t* status, uint32_t* sched, int num_sms, cudaStream_t st) {
  // the shared-memory opt-in, once per device (host threads may race here)
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      err = cudaFuncSetAttribute(mxfp4_gemm_kernel<kMode, kTok>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 Cfg<kTok>::ALLOC);
      if (err != cudaSuccess) return err;
      if (dev < 64) done[dev] = true;
    }
  }
  const int K = kMode == kDown ? s.I : s.H;
  const int N_out = kMode == kDown ? s.H : s.I;
  const int NT = kMode == kDown ? (N_out + 255) / 256 : N_out / 128;
  const int64_t R = static_cast<int64_t>(s.T) * s.k;
  const int64_t max_tiles = (R / kTok + (s.E < R ? s.E : R)) * NT;
  if (num_sms > kMaxDrawers) num_sms = kMaxDrawers;
  const int grid = static_cast<int>(max_tiles < num_sms ? max_tiles : num_sms);
  return launch_pdl(mxfp4_gemm_kernel<kMode, kTok>, dim3(grid), dim3(Cfg<kTok>::THREADS), Cfg<kTok>::ALLOC, st, m,
                    sfT, sfW0, sfW1, D, Dsf, off_pad, counts, s.E, K, N_out, NT, max_rows_of(s), status, sched);
}

// Windows of 128 rows leave shared memory for a fourth stage, and their ten
// warps registers for the whole accumulators; windows of 192 read the weights
// less often.  Measured (gate/up | down, us, 4096 x 1536, 64 experts): 8 rows per
// expert 71 | 36 with 128 and 76 | 37 with 192, 256 rows 107 | 73 and 114 | 74,
// 320 rows 125 | 85 and 121 | 80, 512 rows 173 | 121 and 164 | 110.
constexpr int kWideRows = 256;  // rows per expert, on average, above which windows have 192

template <int kMode, typename... Args>
cudaError_t launch(const moe_shape& s, Args... args) {
  const bool wide = static_cast<int64_t>(s.T) * s.k > static_cast<int64_t>(kWideRows) * s.E;
  return wide ? launch_tok<kMode, 192>(s, args...) : launch_tok<kMode, 128>(s, args...);
}

}  // namespace

cudaError_t launch_mxfp4_up(const moe_shape& s, const Mxfp4Maps& m, const uint8_t* x_scales, const uint8_t* wg_scales,
                            const uint8_t* wu_scales, uint16_t* h, const int32_t* off_pad, const int32_t* counts,
                            uint32_t* status, uint32_t* sched, int num_sms, cudaStream_t st) {
  return launch<kUpBf16>(s, m, x_scales, wg_scales, wu_scales, h, nullptr, off_pad, counts, status, sched, num_sms, st);
}

cudaError_t launch_mxfp4_up_quantized(const moe_shape& s, const Mxfp4Maps& m, const uint8_t* x_scales,
                                      const uint8_t* wg_scales, const uint8_t* wu_scales, uint8_t* h_codes,
                                      uint8_t* h_scales, const int32_t* off_pad, const int32_t* counts,
                                      uint32_t* status, uint32_t* sched, int num_sms, cudaStream_t st) {
  return launch<kUpMxfp4>(s, m, x_scales, wg_scales, wu_scales, h_codes, h_scales, off_pad, counts, status, sched,
                          num_sms, st);
}

cudaError_t launch_mxfp4_down(const moe_shape& s, const Mxfp4Maps& m, const uint8_t* h_scales,
                              const uint8_t* wd_scales, uint16_t* Y, const int32_t* off_pad, const int32_t* counts,
                              uint32_t* status, uint32_t* sched, int num_sms, cudaStream_t st) {
  return launch<kDown>(s, m, h_scales, wd_scales, wd_scales, Y, nullptr, off_pad, counts, status, sched, num_sms, st);
}

}  // namespace moe
