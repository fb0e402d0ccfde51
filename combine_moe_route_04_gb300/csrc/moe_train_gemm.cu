// moe_train_gemm.cu -- grouped products of the experts' backward pass
// (tcgen05, two-CTA MMAs).
//
// With g = X Wg, u = X Wu, s = sigmoid(g), h = g s u, Y = h Wd per expert:
//   down backward:   dh = dY Wd^T, dg = dh u s (1 + g (1 - s)), du = dh g s
//   up backward:     dX = dg Wg^T + du Wu^T (one reduction of length 2 I)
//   weight backward: dWg = X^T dg, dWu = X^T du, dWd = h^T dY
// Every product is out[n, m] = sum_k B[n, k] A[m, k], m the contiguous axis of
// the output: rows of an expert (n) times weight rows (m), both with k
// contiguous, in the first two; columns of X or h (n) times columns of the
// gradients (m), k running over the expert's rows, in the third, whose operands
// both have k as their outer axis.
//
// A cluster of two CTAs computes a tile of 256 m x up to 256 n (M = 256 MMAs,
// cta_group::2; CTA r holds 128 of the m and supplies half of the n) into one
// of two accumulators of 256 TMEM columns, so that the epilogue of a tile runs
// under the next one's MMAs.  TMEM lane = m, column = n: a piece of 32 n x 128
// m is rounded to bf16, transposed through shared memory (stmatrix) and stored
// by TMA.  In the down backward the same piece of g and u is loaded into that
// staging first and read with ldmatrix, which gives each thread the elements
// whose dh it holds; dg and du go back to the same places.
//
// The reduction of the weight backward ends inside a 16-row step of the MMA when
// an expert's count is no multiple of 16, and the padding rows behind it may
// hold anything.  The last stage of such a tile completes on a barrier of its
// own CTA; a warp then clears the rows behind the last one in shared memory and
// hands the stage on.
#include <cstdint>
#include <mutex>

#include "moe_device.cuh"
#include "moe_internal.h"
#include "moe_transpose.cuh"

namespace moe {
namespace {

enum Mode { kDownBwd = 0, kUpBwd = 1, kWeightBwd = 2 };

constexpr int kMaxExperts = 256;
constexpr int kStageK = 64;               // reduction elements per stage
constexpr int kTileM = 256;               // output columns per tile (128 per CTA)
constexpr int kTileN = 256;               // most output rows per tile
constexpr int kOperandBytes = 128 * kStageK * 2;  // 128 m (or n) x 64 k
constexpr int kStageBytes = 2 * kOperandBytes;
constexpr int kBoxBytes = kStageK * 128;  // 64 k x 64 columns (weight backward)
constexpr int kEpiWarps = 8;              // two per TMEM lane quarter, taking 32-row pieces in turn
constexpr int kTurns = kEpiWarps / 4;
constexpr int kTileRing = 8;              // tile indices on their way from the scheduler
constexpr uint32_t kTmemCols = 512;

template <int kMode>
struct Cfg {
  static constexpr int FIX_WARPS = kMode == kWeightBwd ? 1 : 0;
  static constexpr int THREADS = (2 + kEpiWarps + FIX_WARPS) * 32;
  // readers of a tile index: CTA 0's MMA lane and CTA 1's producer lane, both
  // CTAs' epilogue (and clearing) warps
  static constexpr int READERS = 2 + 2 * (kEpiWarps + FIX_WARPS);
  static constexpr int STAGES = kMode == kDownBwd ? 5 : 6;
  // staging per turn: dg and du (32 rows x 128 columns each), or one output piece
  static constexpr int PIECES = kMode == kDownBwd ? 2 : 1;
  static constexpr int OUT_OFF = STAGES * kStageBytes;
  static constexpr int BAR_OFF = OUT_OFF + kTurns * PIECES * kPieceBytes;
  // full, empty, tail, cleared [STAGES]; tfull, tempty [2]; inputs [kTurns];
  // drain; ring full, empty [kTileRing]
  static constexpr int NUM_BARS = 4 * STAGES + 4 + kTurns + 1 + 2 * kTileRing;
  static constexpr int SLOT_OFF = BAR_OFF + NUM_BARS * 8;
  static constexpr int TILE_OFF = SLOT_OFF + 16;
  static constexpr int WIN_OFF = TILE_OFF + kTileRing * 4;
  static constexpr int CNT_OFF = WIN_OFF + (kMaxExperts + 1) * 4;
  static constexpr int OFFP_OFF = CNT_OFF + kMaxExperts * 4;
  static constexpr int BYTES = OFFP_OFF + (kMaxExperts + 1) * 4;
  static constexpr int ALLOC = BYTES + 1024;
  static_assert(ALLOC <= 232448, "shared memory budget");
};

struct Tile {
  int e;     // expert
  int mat;   // weight backward: gate, up, down
  int m0;    // first output column of the pair
  int n0;    // first row: of the window, or of the expert's gradient matrix
  int n;     // real rows (1..256)
  int k;     // length of the reduction
  bool ok;
};

struct Problem {
  int E, H, I;
  int64_t max_rows;
};

// Down and up backward: an expert's c rows are cut into nw = ceil(c / 256)
// windows of equal size (rounded up to 16), so that those which share a weight
// tile run in step; tile = expert, then column tile, then window.
// Weight backward: tile = expert, then gate / up / down, then row tile, then
// column tile.
template <int kMode>
__device__ __forceinline__ Tile decode(int tile, const Problem& p, const int32_t* win, const int32_t* offp,
                                       const int32_t* cnt) {
  Tile c{0, 0, 0, 0, 0, 0, false};
  if constexpr (kMode == kWeightBwd) {
    const int ti = (p.I + 255) / 256, th = (p.H + 255) / 256;
    const int per = ti * th;
    c.e = tile / (3 * per);
    if (c.e >= p.E) return c;
    const int rem = tile - c.e * 3 * per;
    c.mat = rem / per;
    const int at = rem - c.mat * per;
    const int tm = c.mat == 2 ? th : ti;  // column tiles
    c.m0 = at % tm * kTileM;
    c.n0 = at / tm * kTileN;
    c.n = min(kTileN, (c.mat == 2 ? p.I : p.H) - c.n0);
    c.k = cnt[c.e];
  } else {
    const int nt = ((kMode == kDownBwd ? p.I : p.H) + 255) / 256;
    const int q = tile / nt;
    int lo = 0, hi = p.E;  // last e with win[e] <= q
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (win[mid] <= q) lo = mid; else hi = mid - 1;
    }
    if (lo >= p.E) return c;
    const int nw = win[lo + 1] - win[lo];
    const int local = tile - nt * win[lo];
    if (nw <= 0 || local < 0 || local >= nt * nw) return c;
    const int w = local % nw;
    const int size = ((cnt[lo] + nw - 1) / nw + 15) / 16 * 16;
    c.e = lo;
    c.m0 = local / nw * kTileM;
    c.n = min(size, cnt[lo] - size * w);
    c.n0 = size * w;  // relative to the expert's first row until checked
    c.k = kMode == kDownBwd ? p.H : 2 * p.I;
  }
  // the expert's rows lie inside its 128-row blocks, and those inside the buffers
  const int64_t first = offp[c.e], end = offp[c.e + 1];
  const int rows = cnt[c.e];
  c.ok = c.n > 0 && c.n <= kTileN && rows >= 0 && first >= 0 && first + rows <= end && end <= p.max_rows;
  if (kMode != kWeightBwd) c.n0 += static_cast<int>(first);
  return c;
}

// Tiles are drawn from a counter in the workspace, in order: cluster b starts
// on tile b, and CTA 0's producer lane publishes every later index to both CTAs
// a whole tile before it is needed.  The cluster that stops drawing last clears
// the counter, and knows whether the launch started from a cleared one: the word
// behind it counts the clusters that have stopped (bits 0-9), sums their indexes
// plus one (bits 10-29), and gets bit 30 from the one that drew 0.  With anything
// else in either word the sum comes out wrong (tiles may have been left out).
constexpr int kMaxClusters = 1023;
__device__ __forceinline__ uint32_t stopped(uint32_t clusters, uint32_t index_sum, bool drew_zero) {
  return clusters | (index_sum << 10) | (drew_zero ? 1u << 30 : 0u);
}
struct TileRing {
  uint64_t* full;         // [kTileRing], this CTA: one arrival (the scheduler)
  uint64_t* empty;        // [kTileRing], used in CTA 0: READERS arrivals
  volatile int32_t* idx;  // [kTileRing], this CTA
};
__device__ __forceinline__ bool ring_put(const TileRing& r, uint32_t n, int tile, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  if (!mbar_wait<true>(&r.empty[slot], ((n / kTileRing) & 1u) ^ 1u, abort, status)) return false;
  r.idx[slot] = tile;
  mbar_arrive(&r.full[slot]);
  const uint32_t there = map_to_cta(const_cast<int32_t*>(&r.idx[slot]), 1);
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(there), "r"(tile) : "memory");
  mbar_arrive_cluster(map_to_cta(&r.full[slot], 1));
  return true;
}
// The n-th tile of this cluster, -1 when the wait gave up; released at once.
__device__ __forceinline__ int ring_peek(const TileRing& r, uint32_t n, uint32_t rank, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  const uint32_t ph = (n / kTileRing) & 1u;
  const bool ok = rank == 0 ? mbar_wait<false>(&r.full[slot], ph, abort, status)
                            : mbar_wait<true>(&r.full[slot], ph, abort, status);
  return ok ? r.idx[slot] : -1;
}
__device__ __forceinline__ void ring_release(const TileRing& r, uint32_t n, uint32_t rank, uint32_t empty0) {
  const uint32_t slot = n % kTileRing;
  if (rank == 0) mbar_arrive(&r.empty[slot]);
  else mbar_arrive_cluster(empty0 + 8u * slot);
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

// dg and du of one element.  The sigmoid is formed on the SFU (relative error
// about |g| 2^-24 and a few ulps below zero, far under the outputs' rounding to
// bf16); where exp(-g) is infinite, s is 0 and both are 0.
__device__ __forceinline__ void swiglu_backward(float dh, float g, float u, float& dg, float& du) {
  const float s = __fdividef(1.0f, 1.0f + __expf(-g));
  const float gs = g * s;
  du = dh * gs;
  dg = dh * u * (s + gs * (1.0f - s));
}

template <int kMode>
__global__ void __launch_bounds__(Cfg<kMode>::THREADS, 1)
    train_gemm_kernel(const __grid_constant__ TrainMaps maps, uint16_t* __restrict__ D0, uint16_t* __restrict__ D1,
                      const int32_t* __restrict__ off_pad, const int32_t* __restrict__ counts, Problem p,
                      uint32_t* __restrict__ status, uint32_t* __restrict__ sched) {
  using C = Cfg<kMode>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tail = empty + C::STAGES;      // this CTA's loads of a stage that is to be cleared
  uint64_t* cleared = tail + C::STAGES;    // used in CTA 0: CTA 1 has cleared its part
  uint64_t* tfull = cleared + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* inbar = tempty + 2;            // [kTurns] g and u of a piece
  uint64_t* drain = inbar + kTurns;
  const TileRing ring{drain + 1, drain + 1 + kTileRing, reinterpret_cast<volatile int32_t*>(smem + C::TILE_OFF)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int32_t* s_win = reinterpret_cast<int32_t*>(smem + C::WIN_OFF);
  int32_t* s_cnt = reinterpret_cast<int32_t*>(smem + C::CNT_OFF);
  int32_t* s_offp = reinterpret_cast<int32_t*>(smem + C::OFFP_OFF);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: draws the tiles and issues the MMAs

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
      mbar_init(&cleared[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    for (int t = 0; t < kTurns; ++t) mbar_init(&inbar[t], 1);
    mbar_init(drain, 1);
    for (int i = 0; i < kTileRing; ++i) {
      mbar_init(&ring.full[i], 1);
      mbar_init(&ring.empty[i], C::READERS);
    }
    *abort_flag = 0;
    fence_mbarrier_init();
    prefetch_tmap(&maps.a[0]);
    prefetch_tmap(&maps.b[0][0]);
    prefetch_tmap(&maps.out[0]);
  }
  cluster_sync_all();  // both CTAs' barriers exist before any cross-CTA arrival
  if (warp == 1) {
    tmem_alloc_pair(tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();
  if (warp == 2) {
    // windows per expert -> exclusive scan (E <= 256)
    constexpr int per = kMaxExperts / 32;
    int loc[per];
    int sum = 0;
#pragma unroll
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      int nw = 0;
      if (e < p.E) {
        int c = __ldcg(counts + e);
        if (c > p.max_rows) {  // no buffer holds so many: no tiles for them
          record_status(status, kStatusBounds);
          c = kMode == kWeightBwd ? -1 : 0;
        }
        s_cnt[e] = c;
        nw = c > 0 ? (c - 1) / kTileN + 1 : 0;
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
      if (e <= p.E) s_win[e] = run;
      run += loc[i];
    }
    if (lane == 31 && 32 * per == p.E) s_win[p.E] = incl;
  } else if (warp == 3) {
    for (int e = lane; e <= p.E; e += 32) s_offp[e] = __ldcg(off_pad + e);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int total;
  if constexpr (kMode == kWeightBwd) {
    total = p.E * 3 * ((p.I + 255) / 256) * ((p.H + 255) / 256);
  } else {
    // windows of counts that fit the buffers (see the check of each window):
    // nw windows hold more than 256 (nw - 1) rows
    const bool fits = static_cast<int64_t>(s_win[p.E] - p.E) * kTileN <= p.max_rows;
    if (!fits && threadIdx.x == 0) record_status(status, kStatusBounds);
    total = fits ? ((kMode == kDownBwd ? p.I : p.H) + 255) / 256 * s_win[p.E] : 0;
  }
  const uint32_t nclusters = gridDim.x >> 1;
  const uint32_t cluster = blockIdx.x >> 1;
  const uint32_t full0 = map_to_cta(full, 0);
  const uint32_t tempty0 = map_to_cta(tempty, 0);
  const uint32_t rempty0 = map_to_cta(ring.empty, 0);
  auto stages_of = [](int k) { return (k + kStageK - 1) / kStageK; };
  // the last stage of a reduction that ends inside a 16-deep step
  auto has_tail = [](const Tile& c) { return kMode == kWeightBwd && (c.k & 15) != 0; };

  if (warp == 0) {
    // ---------------------------------------------------------- loads (both CTAs)
    if (elect_one_sync()) {
      const uint64_t pol_keep = policy_evict_last();
      const uint64_t pol_normal = policy_evict_normal();
      const uint64_t pol_once = policy_evict_first();
      uint32_t it = 0;
      bool drew_zero = false;
      bool stop = false;
      int tile = static_cast<int>(cluster);
      uint32_t drawn = 0;
      if (rank == 0) {
        drawn = atomicAdd(sched, 1u);  // tile 1's index
        stop = !ring_put(ring, 0, tile, abort_flag, status);
      } else {
        tile = ring_peek(ring, 0, rank, abort_flag, status);
        if (tile >= 0) ring_release(ring, 0, rank, rempty0);
      }
      for (uint32_t n = 0; !stop && tile >= 0 && tile < total; ++n) {
        int next = total;
        if (rank == 0) {
          drew_zero |= drawn == 0u;
          // a cleared counter gives less than total + 2 clusters here
          const uint64_t t = static_cast<uint64_t>(nclusters) + drawn;
          if (t < static_cast<uint64_t>(total)) next = static_cast<int>(t);
          else if (t >= static_cast<uint64_t>(total) + 2u * nclusters) record_status(status, kStatusBounds);
          if (!ring_put(ring, n + 1, next, abort_flag, status)) {
            stop = true;
            break;
          }
          drawn = atomicAdd(sched, 1u);
        }
        const Tile c = decode<kMode>(tile, p, s_win, s_offp, s_cnt);
        if (!c.ok) record_status(status, kStatusBounds);
        const int nk = c.ok ? stages_of(c.k) : 0;
        const int n_half = (c.n + 15) / 16 * 8;  // output rows this CTA supplies
        const int m_first = c.m0 + 128 * static_cast<int>(rank);
        if constexpr (kMode == kWeightBwd) {
          const CUtensorMap* ma = &maps.a[c.mat];
          const CUtensorMap* mb = &maps.b[c.mat == 2 ? 1 : 0][0];
          const int n_first = c.n0 + n_half * static_cast<int>(rank);  // 64 or 128 columns
          const uint32_t mine = static_cast<uint32_t>(2 + n_half / 64) * kBoxBytes;
          for (int kb = 0; kb < nk; ++kb, ++it) {
            const uint32_t s = it % C::STAGES;
            if (!mbar_wait(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, status)) {
              stop = true;
              break;
            }
            const bool own = kb == nk - 1 && has_tail(c);
            const uint32_t fb = own ? map_to_cta(&tail[s], rank) : full0 + 8u * s;
            if (own) mbar_arrive_expect_tx(&tail[s], mine);
            else if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * mine);
            uint8_t* st = smem + s * kStageBytes;
            const int row = s_offp[c.e] + kb * kStageK;
            tma_load_2d_pair(st, ma, fb, m_first, row, pol_keep);
            tma_load_2d_pair(st + kBoxBytes, ma, fb, m_first + 64, row, pol_keep);
            tma_load_2d_pair(st + kOperandBytes, mb, fb, n_first, row, pol_keep);
            if (n_half > 64) tma_load_2d_pair(st + kOperandBytes + kBoxBytes, mb, fb, n_first + 64, row, pol_keep);
          }
        } else {
          // weights that one window alone reads leave L2 first
          const uint64_t pol_w = s_win[c.e + 1] - s_win[c.e] == 1 ? pol_once : pol_normal;
          const int pick = n_half <= 16 ? 0 : n_half <= 32 ? 1 : n_half <= 64 ? 2 : 3;
          const uint32_t bytes = 2u * (kOperandBytes + train_token_box(pick) * kStageK * 2);
          const int row = c.n0 + n_half * static_cast<int>(rank);
          const int m_row = c.e * (kMode == kDownBwd ? p.I : p.H) + m_first;
          const int half = kMode == kUpBwd ? p.I / kStageK : nk;  // stages of the first term
          for (int kb = 0; kb < nk; ++kb, ++it) {
            const uint32_t s = it % C::STAGES;
            if (!mbar_wait(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, status)) {
              stop = true;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            uint8_t* st = smem + s * kStageBytes;
            const int term = kb >= half ? 1 : 0;
            const int k0 = (kb - term * half) * kStageK;
            tma_load_2d_pair(st, &maps.a[term], full0 + 8u * s, k0, m_row, pol_w);
            tma_load_2d_pair(st + kOperandBytes, &maps.b[term][pick], full0 + 8u * s, k0, row, pol_keep);
          }
        }
        if (stop) break;
        if (rank == 0) {
          tile = next;
        } else {
          tile = ring_peek(ring, n + 1, rank, abort_flag, status);
          if (tile >= 0) ring_release(ring, n + 1, rank, rempty0);
        }
      }
      if (rank == 0) {
        drew_zero |= drawn == 0u;
        __threadfence();
        const uint32_t mine = stopped(1u, cluster + 1u, drew_zero);
        const uint32_t seen = atomicAdd(sched + 1, mine) + mine;
        if ((seen & 0x3FFu) == nclusters) {  // every cluster has drawn its last index
          if (seen != stopped(nclusters, nclusters * (nclusters + 1u) / 2u, true))
            record_status(status, kStatusBounds);
          atomicExch(sched, 0u);
          atomicExch(sched + 1, 0u);
        }
      }
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
    // ---------------------------------------------------------- MMAs (CTA 0)
    if (rank == 0 && elect_one_sync()) {
      constexpr bool kOuterK = kMode == kWeightBwd;  // k is the operands' outer axis
      constexpr uint32_t idesc_base = (1u << 4) | (1u << 7) | (1u << 10) | (kOuterK ? 3u << 15 : 0u) |
                                      ((256u >> 4) << 24);
      uint32_t it = 0;
      uint32_t tcount = 0;
      bool stop = false;
      for (uint32_t n = 0; !stop; ++n) {
        const int tile = ring_peek(ring, n, rank, abort_flag, status);
        if (tile < 0 || tile >= total) break;
        ring_release(ring, n, rank, rempty0);
        const Tile c = decode<kMode>(tile, p, s_win, s_offp, s_cnt);
        if (!c.ok || c.k == 0) continue;
        const uint32_t idesc = idesc_base | ((static_cast<uint32_t>(c.n + 15) / 16 * 2) << 17);
        const uint32_t a = tcount & 1u;
        if (!mbar_wait<true>(&tempty[a], ((tcount >> 1) & 1u) ^ 1u, abort_flag, status)) break;
        tc_fence_after();
        const uint32_t d = tmem + a * kTileN;
        const int nk = stages_of(c.k);
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const uint32_t s = it % C::STAGES;
          if (!mbar_wait<true>(&full[s], (it / C::STAGES) & 1u, abort_flag, status)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t sa = smem_u32(smem + s * kStageBytes);
          const uint32_t sb = sa + kOperandBytes;
          if constexpr (kOuterK) {
            // 64-column boxes 8 KB apart, 8-row groups 1 KB apart, a step of 16 rows 2 KB
            const int steps = min(kStageK, c.k - kb * kStageK + 15) / 16;
            for (int kk = 0; kk < steps; ++kk)
              tc_mma_f16_pair(d, smem_desc(sa + kk * 2048, kBoxBytes, 1024, kSwizzle128B),
                              smem_desc(sb + kk * 2048, kBoxBytes, 1024, kSwizzle128B), idesc,
                              (kb | kk) != 0 ? 1u : 0u);
          } else {
#pragma unroll
            for (int kk = 0; kk < kStageK / 16; ++kk)
              tc_mma_f16_pair(d, smem_desc(sa + kk * 32, 16, 1024, kSwizzle128B),
                              smem_desc(sb + kk * 32, 16, 1024, kSwizzle128B), idesc, (kb | kk) != 0 ? 1u : 0u);
          }
          tc_commit_pair(&empty[s], 0x3);
        }
        if (stop) break;
        tc_commit_pair(&tfull[a], 0x3);
        ++tcount;
      }
      tc_commit_pair(drain, 0x1);
      int no_abort = 0;
      mbar_wait(drain, 0, &no_abort, status);
    }
    __syncwarp();
  } else if (warp < 2 + kEpiWarps) {
    // ---------------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3;
    const int turn = (warp - 2) / 4;
    uint8_t* out = smem + C::OUT_OFF + turn * C::PIECES * kPieceBytes;
    const uint32_t out_addr = smem_u32(out);
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    const bool leader = q == 0 && lane == 0;  // of the turn's four warps: TMA
    const int N_out = kMode == kDownBwd ? p.I : p.H;  // (weight backward: the output is never partial)
    uint32_t tcount = 0;
    uint32_t loads = 0;  // pieces of g and u asked for
    for (uint32_t n = 0;; ++n) {
      const int tile = ring_peek(ring, n, rank, abort_flag, status);
      __syncwarp();
      if (lane == 0) ring_release(ring, n, rank, rempty0);
      bool ok = tile >= 0;
      const bool real = ok && tile < total;
      const Tile c = decode<kMode>(real ? tile : 0, p, s_win, s_offp, s_cnt);
      const uint32_t a = tcount & 1u;
      const int col0 = c.m0 + 128 * static_cast<int>(rank);
      const int cols = kMode == kWeightBwd ? (c.mat == 2 ? p.H : p.I) : N_out;
      const bool mine = real && c.ok && col0 < cols;  // this CTA has columns to write
      const int pieces = (c.n + 31) / 32;
      // g and u of piece pc, loaded to where dg and du will be staged
      auto ask = [&](int pc) {
        if (leader) {
          tma_store_wait_read<0>();
          mbar_arrive_expect_tx(&inbar[turn], 2 * kPieceBytes);
          const int r = c.n0 + pc * 32;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            tma_load_2d(out + i * kPieceBytes, &maps.in[i], &inbar[turn], col0, r, policy_evict_first());
            tma_load_2d(out + i * kPieceBytes + kPieceBytes / 2, &maps.in[i], &inbar[turn], col0 + 64, r,
                        policy_evict_first());
          }
        }
        ++loads;
      };
      const bool early = kMode == kDownBwd && mine && turn < pieces;
      if (early) ask(turn);
      if (real && c.ok && c.k > 0) ok = mbar_wait<true>(&tfull[a], (tcount >> 1) & 1u, abort_flag, status);
      if (vote_any(!ok)) {  // every warp gives up together (they share barriers)
        if (early && leader) {
          int no_abort = 0;
          mbar_wait(&inbar[turn], (loads - 1) & 1u, &no_abort, status);
        }
        break;
      }
      if (tile >= total) break;
      if (!c.ok) continue;
      tc_fence_after();
      if (c.k > 0) ++tcount;
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8u * a);
      };
      // the output pieces in the staging leave: 32 full rows by TMA, fewer by
      // the warps, eight rows each, sixteen lanes a row
      auto store = [&](int pc) {
        fence_proxy_async_smem();
        named_barrier_sync(3 + turn, 128);
        const int left = c.n - pc * 32;
        const int r0 = (kMode == kWeightBwd ? c.e * (c.mat == 2 ? p.I : p.H) : 0) + c.n0 + pc * 32;
        if (left >= 32) {
          if (leader) {
#pragma unroll
            for (int i = 0; i < C::PIECES; ++i) {
              const CUtensorMap* m = kMode == kWeightBwd ? &maps.out[c.mat] : &maps.out[i];
              tma_store_2d(m, out + i * kPieceBytes, col0, r0);
              tma_store_2d(m, out + i * kPieceBytes + kPieceBytes / 2, col0 + 64, r0);
            }
            tma_store_commit();
          }
          __syncwarp();
          return;
        }
#pragma unroll
        for (int i = 0; i < C::PIECES; ++i) {
          uint16_t* D = i == 0 ? D0 : D1;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = 8 * q + 2 * j + (lane >> 4);
            if (t < left)
              *reinterpret_cast<uint4*>(D + static_cast<int64_t>(r0 + t) * N_out + col0 + (lane & 15) * 8) =
                  *reinterpret_cast<const uint4*>(out + i * kPieceBytes + staged_at(t, lane & 15));
          }
        }
        named_barrier_sync(3 + turn, 128);  // read before the next piece arrives
      };
      const int count = pieces > turn ? (pieces - turn + kTurns - 1) / kTurns : 0;  // this turn's pieces
      if (!mine || count == 0) {
        if (c.k > 0) release();
        continue;
      }
      for (int i = 0; i < count; ++i) {
        const int pc = turn + kTurns * i;
        uint32_t v[32];
        if (kMode != kWeightBwd || c.k > 0) {
          load_piece(tb + a * kTileN + pc * 32, v);
          tmem_ld_wait();
          if (i == count - 1) release();
        } else {  // an expert without rows: its gradient is zero
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0u;
        }
        if constexpr (kMode == kDownBwd) {
          bool in = mbar_wait(&inbar[turn], (loads - 1) & 1u, abort_flag, status);
          (void)in;  // (a wait that gave up has raised the abort flag: the values are not used)
          const uint32_t at = out_addr + staged_at(lane & 7, 4 * q + (lane >> 3));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t g[4], u[4];
            ldmatrix_x4_trans(at + 8 * j * 128, g);
            ldmatrix_x4_trans(at + kPieceBytes + 8 * j * 128, u);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int k = piece_entry(4 * j + x);
              float dg0, du0, dg1, du1;
              swiglu_backward(__uint_as_float(v[k]), bf16lo_to_f32(g[x]), bf16lo_to_f32(u[x]), dg0, du0);
              swiglu_backward(__uint_as_float(v[k + 1]), bf16hi_to_f32(g[x]), bf16hi_to_f32(u[x]), dg1, du1);
              g[x] = pack_bf16x2(dg0, dg1);
              u[x] = pack_bf16x2(du0, du1);
            }
            __syncwarp();
            stmatrix_x4_trans(at + 8 * j * 128, g[0], g[1], g[2], g[3]);
            stmatrix_x4_trans(at + kPieceBytes + 8 * j * 128, u[0], u[1], u[2], u[3]);
          }
        } else {
          uint32_t packed[16];
          round_piece(v, packed);
          if (leader) tma_store_wait_read<0>();
          __syncwarp();
          named_barrier_sync(3 + turn, 128);  // the previous piece has been read
          stage_piece(out_addr, q, packed, lane);
        }
        store(pc);
        if (kMode == kDownBwd && i + 1 < count) ask(pc + kTurns);
      }
    }
    if (leader) tma_store_wait_all<0>();  // this thread's stores are written
    __syncwarp();
  } else if constexpr (kMode == kWeightBwd) {
    // ---------------------------------------------------------- clearing (both CTAs)
    uint32_t it = 0;
    uint32_t phases = 0;  // bit s: parity of the next use of stage s's barriers
    for (uint32_t n = 0;; ++n) {
      const int tile = ring_peek(ring, n, rank, abort_flag, status);
      __syncwarp();
      if (tile < 0) break;
      if (lane == 0) ring_release(ring, n, rank, rempty0);
      if (tile >= total) break;
      const Tile c = decode<kMode>(tile, p, s_win, s_offp, s_cnt);
      if (!c.ok) continue;
      it += stages_of(c.k);
      if (!has_tail(c)) continue;
      const uint32_t s = (it - 1) % C::STAGES;
      const uint32_t ph = (phases >> s) & 1u;
      phases ^= 1u << s;
      if (__any_sync(0xffffffffu, !mbar_wait(&tail[s], ph, abort_flag, status))) break;
      const int first = c.k & (kStageK - 1), last = (first + 15) & ~15;
      // lane: box (two of each operand, or one of the second) and 16-byte chunk
      uint8_t* box = smem + s * kStageBytes + (lane >> 3) * kBoxBytes + (lane & 7) * 16;
      for (int r = first; r < last; ++r) *reinterpret_cast<uint4*>(box + r * 128) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      bool ok = true;
      if (lane == 0) {
        if (rank == 0) {
          ok = mbar_wait<true>(&cleared[s], ph, abort_flag, status);
          if (ok) mbar_arrive(&full[s]);
        } else {
          mbar_arrive_cluster(map_to_cta(&cleared[s], 0));
        }
      }
      if (__any_sync(0xffffffffu, !ok)) break;
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) {
    __syncwarp();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <int kMode>
cudaError_t launch(const moe_shape& s, const TrainMaps& m, uint16_t* D0, uint16_t* D1, const int32_t* off_pad,
                   const int32_t* counts, uint32_t* status, uint32_t* sched, int num_sms, cudaStream_t st) {
  using C = Cfg<kMode>;
  // the shared-memory opt-in, once per device (host threads may race here)
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      err = cudaFuncSetAttribute(train_gemm_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::ALLOC);
      if (err != cudaSuccess) return err;
      if (dev < 64) done[dev] = true;
    }
  }
  const int64_t ti = (s.I + 255) / 256, th = (s.H + 255) / 256;
  int64_t tiles;
  if (kMode == kWeightBwd) tiles = s.E * 3 * ti * th;
  else tiles = max_windows_of(s) * (kMode == kDownBwd ? ti : th);
  int64_t clusters = num_sms / 2;
  if (clusters > kMaxClusters) clusters = kMaxClusters;
  if (tiles < clusters) clusters = tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::ALLOC;
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
  return cudaLaunchKernelEx(&cfg, train_gemm_kernel<kMode>, m, D0, D1, off_pad, counts,
                            Problem{s.E, s.H, s.I, max_rows_of(s)}, status, sched);
}

}  // namespace

cudaError_t launch_down_backward(const moe_shape& s, const TrainMaps& m, uint16_t* dg, uint16_t* du,
                                 const int32_t* off_pad, const int32_t* counts, uint32_t* status, uint32_t* sched,
                                 int num_sms, cudaStream_t st) {
  return launch<kDownBwd>(s, m, dg, du, off_pad, counts, status, sched, num_sms, st);
}

cudaError_t launch_up_backward(const moe_shape& s, const TrainMaps& m, uint16_t* dx, const int32_t* off_pad,
                               const int32_t* counts, uint32_t* status, uint32_t* sched, int num_sms,
                               cudaStream_t st) {
  return launch<kUpBwd>(s, m, dx, nullptr, off_pad, counts, status, sched, num_sms, st);
}

cudaError_t launch_weight_backward(const moe_shape& s, const TrainMaps& m, const int32_t* off_pad,
                                   const int32_t* counts, uint32_t* status, uint32_t* sched, int num_sms,
                                   cudaStream_t st) {
  return launch<kWeightBwd>(s, m, nullptr, nullptr, off_pad, counts, status, sched, num_sms, st);
}

}  // namespace moe
