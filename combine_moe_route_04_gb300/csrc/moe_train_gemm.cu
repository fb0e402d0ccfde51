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
// under the next one's MMAs.  TMEM lane = m, column = n: a piece of 64 n x 128
// m is rounded to bf16, transposed through shared memory (stmatrix) and stored
// by TMA.  In the down backward pieces have 32 n, and the same piece of g and u is
// loaded into that staging first and read with ldmatrix, which gives each thread
// the elements whose dh it holds; dg and du go back to the same places.
//
// In the weight backward a cluster takes a run of column tiles over the same rows of
// a gradient matrix, and where the reduction's stages of the second operand all have
// room (STAGES), they stay for the run's tiles: half the traffic from L2.
//
// What bounds it (64 experts of 4096 x 1536, 256 rows each): the down and up backward
// HBM, 1.14 GB in 215 us and 1.85 GB in 324 us (5.3 and 5.7 TB/s; with 8 rows per
// expert 6.0 and 7.0); the weight backward, 2.4 GB of gradients and 0.6 PFLOP, 520 to
// 565 us, the power cap (1.7 GHz and 1370 W when run on and on); with 8 rows per expert
// 384 us, HBM (6.3 TB/s); with 1000 rows 1650 us, 1.50 PFLOP/s.  One dense block of 5003
// rows, 2176 x 5760: 93 to 114 + 174 + 243 us, 1.1 to 1.35, 1.4 and 1.55 PFLOP/s (the
// down backward's pieces: g and u of one are asked for when the one before has left).
//
// The reduction of the weight backward ends inside a 16-row step of the MMA when
// an expert's count is no multiple of 16, and the padding rows behind it may
// hold anything.  The last stage of such a tile completes on a barrier of its
// own CTA; a warp then clears the rows behind the last one in shared memory and
// hands the stage on.
#include <cstdint>
#include <mutex>

#include "moe_device.cuh"
#include "moe_epilogue.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

enum Mode { kDownBwd = 0, kUpBwd = 1, kWeightBwd = 2 };

constexpr int kMaxExperts = 256;
constexpr int kStageK = 64;               // reduction elements per stage
constexpr int kTileM = 256;               // output columns per tile (128 per CTA)
constexpr int kTileN = 256;               // most output rows per tile
constexpr int kOperandBytes = 128 * kStageK * 2;  // 128 m (or n) x 64 k
constexpr int kBoxBytes = kStageK * 128;  // 64 k x 64 columns (weight backward)
constexpr int kEpiWarps = 8;              // two per TMEM lane quarter, taking 32-row pieces in turn
constexpr int kTurns = kEpiWarps / 4;
constexpr int kTileRing = 8;              // most tiles on their way from the scheduler
constexpr uint32_t kTmemCols = 512;
// warps: loads, MMAs, epilogue, scheduler, clearing (weight backward)
constexpr int kSchedWarp = 2 + kEpiWarps;

template <int kMode>
struct Cfg {
  static constexpr int FIX_WARPS = kMode == kWeightBwd ? 1 : 0;
  static constexpr int THREADS = (3 + kEpiWarps + FIX_WARPS) * 32;
  // readers of a tile: CTA 0's MMA lane, both CTAs' loading lanes, epilogue and
  // clearing warps
  static constexpr int READERS = 3 + 2 * (kEpiWarps + FIX_WARPS);
  // A turn's staging: dg and du of 32 rows; or 64 output rows, in the weight backward
  // twice, so that one half's store is still being read while the other is written
  // (64 experts of 4096 x 1536, 256 rows each: one buffer of 64 rows and a sixth stage
  // 806 us, one of 128 rows 700; later, with cheaper hand-overs, 588 and with two of 64 560).
  static constexpr int HEIGHT = kTrainStoreRows;
  static constexpr int BUFS = kMode == kWeightBwd ? 2 : 1;
  static constexpr int STAGES = kMode == kWeightBwd ? 5 : 6;
  static constexpr int TURN_BYTES = BUFS * HEIGHT * 256;
  static constexpr int B_OFF = STAGES * kOperandBytes;  // the second operand's slots
  static constexpr int OUT_OFF = 2 * B_OFF;
  static constexpr int RING_OFF = OUT_OFF + kTurns * TURN_BYTES;
  static constexpr int BAR_OFF = RING_OFF + kTileRing * 16;
  // full, empty, tail, cleared, bfree [STAGES]; tfull, tempty [2]; inputs [kTurns];
  // drain; ring full, empty [kTileRing]
  static constexpr int NUM_BARS = 5 * STAGES + 4 + kTurns + 1 + 2 * kTileRing;
  static constexpr int SLOT_OFF = BAR_OFF + NUM_BARS * 8;
  static constexpr int SMEM = SLOT_OFF + 16 + 1024;
  static_assert(SMEM <= 232448, "shared memory budget");
  static_assert(kMode != kDownBwd || 2 * kPieceBytes <= TURN_BYTES, "dg and du of a piece");
};

struct Problem {
  int E, H, I;
  int window;      // most rows of a window (down and up backward)
  // weight backward, over a row tile: lengths and numbers of the runs of dWg's and
  // dWu's column tiles, and of dWd's
  int len_x, runs_x, len_h, runs_h;
  uint32_t ahead;  // tiles handed out ahead
  int64_t max_rows;
};

// A tile as the scheduler hands it out.
struct Tile {
  int e;    // expert
  int mat;  // weight backward: gate, up, down; else: 1 where the expert has one window
  int m0;   // first output column of the pair
  int n0;   // weight backward: first row in the expert's gradient matrix
  int n;    // output rows (1..256)
  int row;  // first row of the window, or (weight backward) of the expert
  int k;    // length of the reduction
  bool ok, last;
  bool load_b, free_b;  // weight backward: brings the second operand, is the last to use it
};
__device__ __forceinline__ int4 pack_tile(const Tile& c) {
  return make_int4(c.n | (c.ok ? 1 << 9 : 0) | (c.last ? 1 << 10 : 0) | (c.mat << 11) | (c.e << 13) |
                       (c.load_b ? 1 << 21 : 0) | (c.free_b ? 1 << 22 : 0),
                   (c.m0 / kTileM) | (c.n0 / kTileN << 16), c.row, c.k);
}
__device__ __forceinline__ Tile unpack_tile(const int4& v) {
  Tile c;
  c.n = v.x & 511;
  c.ok = (v.x >> 9) & 1;
  c.last = (v.x >> 10) & 1;
  c.mat = (v.x >> 11) & 3;
  c.e = (v.x >> 13) & 255;
  c.load_b = (v.x >> 21) & 1;
  c.free_b = (v.x >> 22) & 1;
  c.m0 = (v.y & 0xFFFF) * kTileM;
  c.n0 = (v.y >> 16) * kTileN;
  c.row = v.z;
  c.k = v.w;
  return c;
}

// Tiles go to the clusters in order: cluster b starts on tile b, and a warp of its
// CTA 0 draws every later index from a counter in the workspace, finds the tile
// and hands it to all roles of both CTAs through a ring.
// (Each role finding its tile from the index by itself, with three divisions and
// a search, took 860 of the 6800 cycles that a weight tile of 8 rows had.)
struct TileRing {
  uint64_t* full;   // [kTileRing], this CTA: one arrival (the scheduler)
  uint64_t* empty;  // [kTileRing], used in CTA 0: READERS arrivals
  int4* tile;       // [kTileRing], this CTA
};
// Hands out the n-th tile once every role has taken the one `ahead` (at most
// kTileRing) before it.
__device__ __forceinline__ bool ring_put(const TileRing& r, uint32_t n, uint32_t ahead, const Tile& c,
                                         volatile int* abort, uint32_t* status) {
  const uint32_t slot = n % kTileRing, before = n - ahead;
  if (n >= ahead && !mbar_wait<true>(&r.empty[before % kTileRing], (before / kTileRing) & 1u, abort, status))
    return false;
  const int4 v = pack_tile(c);
  *const_cast<volatile int*>(&r.tile[slot].x) = v.x;
  *const_cast<volatile int*>(&r.tile[slot].y) = v.y;
  *const_cast<volatile int*>(&r.tile[slot].z) = v.z;
  *const_cast<volatile int*>(&r.tile[slot].w) = v.w;
  mbar_arrive(&r.full[slot]);
  send_cluster(map_to_cta(&r.tile[slot], 1), map_to_cta(&r.full[slot], 1), v);
  return true;
}
// The n-th tile of this cluster; false when the wait gave up.
__device__ __forceinline__ bool ring_get(const TileRing& r, uint32_t n, uint32_t rank, Tile& c, volatile int* abort,
                                         uint32_t* status) {
  const uint32_t slot = n % kTileRing;
  const uint32_t ph = (n / kTileRing) & 1u;
  const bool ok = rank == 0 ? mbar_wait<false>(&r.full[slot], ph, abort, status)
                            : mbar_wait<true>(&r.full[slot], ph, abort, status);
  if (!ok) return false;
  const volatile int* w = reinterpret_cast<const volatile int*>(&r.tile[slot]);
  c = unpack_tile(make_int4(w[0], w[1], w[2], w[3]));
  return true;
}
__device__ __forceinline__ void ring_release(const TileRing& r, uint32_t n, uint32_t rank, uint32_t empty0) {
  const uint32_t slot = n % kTileRing;
  if (rank == 0) mbar_arrive(&r.empty[slot]);
  else mbar_arrive_peer(empty0 + 8u * slot);
}

// The scheduler: one warp, lane l knowing the experts l, 32 + l, ...  The first tile
// is handed out before the first draws, whose latency the release to the readers
// would wait for.  (Eight neighbouring experts a lane, and the draws first: 28.2 us
// for the three products of 128 tokens, 256 x 512, 8 experts, in a loop where this
// takes 24.7.)
//   down and up backward: an expert's c rows are cut into ceil(c / window) windows of
//   equal size (rounded up to 16), so that those which share a weight tile run in
//   step; tiles in the order expert, column tile, window.
//   weight backward: what is drawn is a run of column tiles (of dWg and dWu, whose
//   second operand is X, or of dWd, whose second operand is h) over one row tile, so
//   that the second operand is brought once for all of them; order: expert, row tile,
//   run, first of dWg and dWu, then of dWd.  Runs have one tile where the operand's
//   stages do not all stay.
template <int kMode>
__device__ __forceinline__ void schedule(const TileRing& ring, const Problem& p, const int32_t* off_pad,
                                         const int32_t* counts, uint32_t cluster, uint32_t nclusters, int lane,
                                         volatile int* abort, uint32_t* status, uint32_t* sched) {
  constexpr int kGroups = kMaxExperts / 32;  // of 32 experts
  const uint32_t all = 0xffffffffu;
  const int ti = (p.I + kTileM - 1) / kTileM, th = (p.H + kTileM - 1) / kTileM;
  const int col_tiles = kMode == kWeightBwd ? 1 : kMode == kDownBwd ? ti : th;
  auto stays = [](int rows) { return rows <= Cfg<kMode>::STAGES * kStageK; };
  int cnt[kGroups], off[kGroups], end[kGroups];
  int nw[kGroups], incl[kGroups];  // windows (or runs) of the expert, and up to it
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    const int e = 32 * i + lane;
    cnt[i] = off[i] = end[i] = 0;
    if (32 * i < p.E && e < p.E) {
      cnt[i] = __ldcg(counts + e);
      off[i] = __ldcg(off_pad + e);
      end[i] = __ldcg(off_pad + e + 1);
    }
  }
  int windows = 0;
#pragma unroll
  for (int i = 0; i < kGroups; ++i) {
    nw[i] = 0;
    incl[i] = windows;
    if (32 * i < p.E) {
      const int e = 32 * i + lane;
      // an expert whose rows do not lie inside its blocks and the buffers gets no rows
      if (e < p.E && (cnt[i] < 0 || off[i] < 0 || static_cast<int64_t>(off[i]) + cnt[i] > end[i] ||
                      end[i] > p.max_rows)) {
        record_status(status, kStatusBounds);
        cnt[i] = kMode == kWeightBwd ? -1 : 0;
      }
      if constexpr (kMode == kWeightBwd)
        nw[i] = e >= p.E || cnt[i] < 0 ? 0 : stays(cnt[i]) ? th * p.runs_x + ti * p.runs_h : 3 * th * ti;
      else
        nw[i] = cnt[i] <= p.window ? (cnt[i] > 0 ? 1 : 0) : (cnt[i] - 1) / p.window + 1;
      int sum = nw[i];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(all, sum, o);
        if (lane >= o) sum += y;
      }
      incl[i] += sum;
      windows += __shfl_sync(all, sum, 31);
    }
  }
  // windows of counts that fit the buffers: nw of them hold more than window * (nw - 1) rows
  const bool fits = kMode == kWeightBwd || static_cast<int64_t>(windows - p.E) * p.window <= p.max_rows;
  if (!fits && lane == 0) record_status(status, kStatusBounds);
  const int total = fits ? col_tiles * windows : 0;

  // two draws on their way (with one, a short tile's time was the atomic's under
  // the output's traffic)
  uint32_t drawn = 0, later = 0;
  bool drew_zero = false;
  // every draw, of lane 0: a cleared counter gives less than total + 2 clusters
  auto checked = [&](uint32_t d) {
    drew_zero |= d == 0u;
    if (d >= static_cast<uint64_t>(total) + 2u * nclusters) record_status(status, kStatusBounds);
  };
  int tile = static_cast<int>(cluster);
  for (uint32_t n = 0;;) {
    Tile c{0, 0, 0, 0, 0, 0, 0, false, tile >= total, false, false};
    int owner = 0;  // the lane that knows the tile's expert
    int first = 0, len = 1;  // weight backward: the run's first column tile, its tiles
    if (tile < total) {
      const int q = tile / col_tiles;  // (all column tiles of a window's expert lie together)
      int rows = 0, row = 0, parts = 1, at = 0;  // the expert's, and the window's place
      bool found = false;
#pragma unroll
      for (int i = 0; i < kGroups; ++i) {
        if (32 * i < p.E && !found) {
          const uint32_t behind = __ballot_sync(all, incl[i] > q);
          found = behind != 0u;
          if (found) {
            owner = __ffs(behind) - 1;
            c.e = 32 * i + lane;
            rows = cnt[i];
            row = off[i];
            parts = nw[i];
            at = tile - col_tiles * (incl[i] - nw[i]);
          }
        }
      }
      c.ok = lane == owner;
      if constexpr (kMode == kWeightBwd) {
        const bool of_x = at < th * (stays(rows) ? p.runs_x : 2 * ti);
        const int a = of_x ? at : at - th * (stays(rows) ? p.runs_x : 2 * ti);
        const int runs = of_x ? (stays(rows) ? p.runs_x : 2 * ti) : stays(rows) ? p.runs_h : th;
        const int most = !stays(rows) ? 1 : of_x ? p.len_x : p.len_h;
        const int panel = a / runs;
        first = (a - panel * runs) * most;
        len = min(most, (of_x ? 2 * ti : th) - first);
        c.mat = of_x ? 0 : 2;
        c.n0 = panel * kTileN;
        c.n = min(kTileN, (of_x ? p.H : p.I) - c.n0);
        c.row = row;
        c.k = rows;
      } else {
        int j = at, w = 0, size = (rows + 15) / 16 * 16;
        if (parts > 1) {
          j = at / parts;
          w = at - j * parts;
          size = ((rows + parts - 1) / parts + 15) / 16 * 16;
        }
        c.mat = parts == 1 ? 1 : 0;
        c.m0 = j * kTileM;
        c.n = min(size, rows - size * w);
        c.row = row + size * w;
        c.k = kMode == kDownBwd ? p.H : 2 * p.I;
        c.ok = c.n > 0;
      }
    }
    bool put = true;
    if (lane == owner) {
      if (kMode == kWeightBwd && !c.last) {
        const bool of_x = c.mat != 2;
        for (int j = 0; j < len && put; ++j) {
          const int m = first + j;
          if (of_x) c.mat = m >= ti ? 1 : 0;
          c.m0 = (c.mat == 1 ? m - ti : m) * kTileM;
          c.load_b = j == 0;
          c.free_b = j == len - 1;
          put = ring_put(ring, n + j, p.ahead, c, abort, status);
        }
      } else {
        put = ring_put(ring, n, p.ahead, c, abort, status);
      }
    }
    if (n == 0 && lane == 0) {
      drawn = atomicAdd(sched, 1u);
      later = atomicAdd(sched, 1u);
    }
    if (__any_sync(all, !put) || tile >= total) break;
    n += kMode == kWeightBwd ? static_cast<uint32_t>(__shfl_sync(all, len, owner)) : 1u;
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

// OR-vote over the threads of a turn of the epilogue (its named barrier).
__device__ __forceinline__ bool vote_any(bool flag, int turn) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pi, po;\n\t"
      "setp.ne.u32 pi, %1, 0;\n\t"
      "bar.red.or.pred po, %3, %2, pi;\n\t"
      "selp.u32 %0, 1, 0, po;\n\t}"
      : "=r"(r)
      : "r"(flag ? 1u : 0u), "n"(kEpiWarps / kTurns * 32), "r"(3 + turn)
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
    train_gemm_kernel(const __grid_constant__ TrainMaps maps, const TrainOut out, const int32_t* __restrict__ off_pad,
                      const int32_t* __restrict__ counts, Problem p, uint32_t* __restrict__ status,
                      uint32_t* __restrict__ sched) {
  using C = Cfg<kMode>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* empty = full + C::STAGES;
  uint64_t* tail = empty + C::STAGES;      // this CTA's loads of a stage that is to be cleared
  uint64_t* cleared = tail + C::STAGES;    // used in CTA 0: CTA 1 has cleared its part
  uint64_t* bfree = cleared + C::STAGES;   // weight backward: a slot of the second operand
  uint64_t* tfull = bfree + C::STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* inbar = tempty + 2;          // [kTurns] g and u of a piece
  uint64_t* drain = inbar + kTurns;
  const TileRing ring{drain + 1, drain + 1 + kTileRing, reinterpret_cast<int4*>(smem + C::RING_OFF)};
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::SLOT_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: schedules and issues the MMAs

  pdl_launch_dependents();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
      mbar_init(&cleared[s], 1);
      mbar_init(&bfree[s], 1);
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
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();
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
      uint32_t it = 0, bit = 0;  // stages so far, and (weight backward) of the second operand
      bool stop = false;
      Tile c;
      for (uint32_t n = 0; !stop && ring_get(ring, n, rank, c, abort_flag, status); ++n) {
        if (c.last) break;
        ring_release(ring, n, rank, rempty0);
        const int nk = c.ok ? stages_of(c.k) : 0;
        const int n_half = (c.n + 15) / 16 * 8;  // output rows this CTA supplies
        const int m_first = c.m0 + 128 * static_cast<int>(rank);
        if constexpr (kMode == kWeightBwd) {
          const CUtensorMap* ma = &maps.a[c.mat];
          const CUtensorMap* mb = &maps.b[c.mat == 2 ? 1 : 0][0];
          const int n_first = c.n0 + n_half * static_cast<int>(rank);  // 64 or 128 columns
          const uint32_t mine = static_cast<uint32_t>(2 + (c.load_b ? n_half / 64 : 0)) * kBoxBytes;
          for (int kb = 0; kb < nk; ++kb, ++it) {
            const uint32_t s = it % C::STAGES, b = bit % C::STAGES;
            if (!mbar_wait(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, status) ||
                (c.load_b && !mbar_wait(&bfree[b], ((bit / C::STAGES) & 1u) ^ 1u, abort_flag, status))) {
              stop = true;
              break;
            }
            const bool own = kb == nk - 1 && has_tail(c);
            const uint32_t fb = own ? map_to_cta(&tail[s], rank) : full0 + 8u * s;
            if (own) mbar_arrive_expect_tx(&tail[s], mine);
            else if (rank == 0) mbar_arrive_expect_tx(&full[s], 2u * mine);
            uint8_t* st = smem + s * kOperandBytes;
            const int row = c.row + kb * kStageK;
            tma_load_2d_pair(st, ma, fb, m_first, row, pol_keep);
            tma_load_2d_pair(st + kBoxBytes, ma, fb, m_first + 64, row, pol_keep);
            if (c.load_b) {
              uint8_t* sb = smem + C::B_OFF + b * kOperandBytes;
              tma_load_2d_pair(sb, mb, fb, n_first, row, pol_keep);
              if (n_half > 64) tma_load_2d_pair(sb + kBoxBytes, mb, fb, n_first + 64, row, pol_keep);
              ++bit;
            }
          }
        } else {
          // weights that one window alone reads leave L2 first
          const uint64_t pol_w = c.mat != 0 ? pol_once : pol_normal;
          const int pick = n_half <= 16 ? 0 : n_half <= 32 ? 1 : n_half <= 64 ? 2 : 3;
          const uint32_t bytes = 2u * (kOperandBytes + train_token_box(pick) * kStageK * 2);
          const int row = c.row + n_half * static_cast<int>(rank);
          const int m_row = c.e * (kMode == kDownBwd ? p.I : p.H) + m_first;
          const int half = kMode == kUpBwd ? p.I / kStageK : nk;  // stages of the first term
          for (int kb = 0; kb < nk; ++kb, ++it) {
            const uint32_t s = it % C::STAGES;
            if (!mbar_wait(&empty[s], ((it / C::STAGES) & 1u) ^ 1u, abort_flag, status)) {
              stop = true;
              break;
            }
            if (rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
            uint8_t* st = smem + s * kOperandBytes;
            const int term = kb >= half ? 1 : 0;
            const int k0 = (kb - term * half) * kStageK;
            tma_load_2d_pair(st, &maps.a[term], full0 + 8u * s, k0, m_row, pol_w);
            tma_load_2d_pair(st + C::B_OFF, &maps.b[term][pick], full0 + 8u * s, k0, row, pol_keep);
          }
        }
      }
      // every stage used must be consumed before the CTA may exit
      const uint32_t nst = it < C::STAGES ? it : C::STAGES;
      for (uint32_t s = 0; s < nst; ++s) {
        const uint32_t last = s + C::STAGES * ((it - 1 - s) / C::STAGES);
        int no_abort = 0;
        mbar_wait(&empty[s], (last / C::STAGES) & 1u, &no_abort, status);
      }
      const uint32_t nb = bit < C::STAGES ? bit : C::STAGES;
      for (uint32_t b = 0; b < nb; ++b) {
        const uint32_t last = b + C::STAGES * ((bit - 1 - b) / C::STAGES);
        int no_abort = 0;
        mbar_wait(&bfree[b], (last / C::STAGES) & 1u, &no_abort, status);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMAs (CTA 0)
    if (rank == 0 && elect_one_sync()) {
      constexpr bool kOuterK = kMode == kWeightBwd;  // k is the operands' outer axis
      constexpr uint32_t idesc_base = (1u << 4) | (1u << 7) | (1u << 10) | (kOuterK ? 3u << 15 : 0u) |
                                      ((256u >> 4) << 24);
      uint32_t it = 0, bit = 0;  // (bit: where the run's second operand starts)
      uint32_t tcount = 0;
      bool stop = false;
      Tile c;
      for (uint32_t n = 0; !stop && ring_get(ring, n, rank, c, abort_flag, status); ++n) {
        if (c.last) break;
        ring_release(ring, n, rank, rempty0);
        if (!c.ok || c.k == 0) continue;
        const uint32_t idesc = idesc_base | ((static_cast<uint32_t>(c.n + 15) / 16 * 2) << 17);
        const uint32_t a = tcount & 1u;
        if (!mbar_wait(&tempty[a], ((tcount >> 1) & 1u) ^ 1u, abort_flag, status)) break;
        tc_fence_after();
        const uint32_t d = tmem + a * kTileN;
        const int nk = stages_of(c.k);
        for (int kb = 0; kb < nk; ++kb, ++it) {
          const uint32_t s = it % C::STAGES;
          if (!mbar_wait(&full[s], (it / C::STAGES) & 1u, abort_flag, status)) {
            stop = true;
            break;
          }
          tc_fence_after();
          const uint32_t b = kOuterK ? (bit + kb) % C::STAGES : s;
          const uint32_t sa = smem_u32(smem + s * kOperandBytes);
          const uint32_t sb = smem_u32(smem + C::B_OFF + b * kOperandBytes);
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
          if (kOuterK && c.free_b) tc_commit_pair(&bfree[b], 0x3);
        }
        if (stop) break;
        if (c.free_b) bit += nk;
        tc_commit_pair(&tfull[a], 0x3);
        ++tcount;
      }
      tc_commit_pair(drain, 0x1);
      int no_abort = 0;
      mbar_wait(drain, 0, &no_abort, status);
    }
    __syncwarp();
  } else if (warp < kSchedWarp) {
    // ---------------------------------------------------------- epilogue (both CTAs)
    const int q = warp & 3;
    const int turn = (warp - 2) / 4;
    const bool leader = q == 0 && lane == 0;  // of the turn's four warps: TMA
    uint8_t* staging = smem + C::OUT_OFF + turn * C::TURN_BYTES;
    const uint32_t tb = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t tcount = 0;
    uint32_t asked = 0;  // pieces of g and u
    for (uint32_t n = 0;; ++n) {
      Tile c{};
      bool ok = ring_get(ring, n, rank, c, abort_flag, status);
      const bool real = ok && !c.last && c.ok;
      const uint32_t a = tcount & 1u;
      const int cols = kMode == kDownBwd ? p.I : kMode == kUpBwd ? p.H : c.mat == 2 ? p.H : p.I;
      const int col0 = c.m0 + 128 * static_cast<int>(rank);
      const int64_t row0 = kMode == kWeightBwd ? static_cast<int64_t>(c.e) * (c.mat == 2 ? p.I : p.H) + c.n0 : c.row;
      const int rows = real && col0 < cols ? c.n : 0;  // (columns are multiples of 128)
      // The turn's four warps: what was staged before has left.
      auto staging_free = [&]() {
        if (leader) tma_store_wait_read<0>();
        __syncwarp();
        named_barrier_sync(3 + turn, 128);
      };
      // They have all staged rows r.. of the tile, `height` of them at most: all by
      // TMA, or fewer by the warps, sixteen lanes a row.
      auto leave = [&](const uint8_t* buf, uint16_t* D, const CUtensorMap* map, int r, int height) {
        const int left = rows - r;
        if (left >= height) {
          if (leader) tma_store_3d(map, buf, 0, static_cast<int32_t>(row0) + r, col0 / 64);
          return;
        }
        for (int t = 2 * q + (lane >> 4); t < left; t += 8)
          *reinterpret_cast<uint4*>(D + (row0 + r + t) * cols + col0 + (lane & 15) * 8) =
              *reinterpret_cast<const uint4*>(buf + staged_at(t, lane & 15, height));
      };
      // g and u of the 32 rows from r, loaded to where dg and du will be staged
      auto ask = [&](int r) {
        if (leader) {
          mbar_arrive_expect_tx(&inbar[turn], 2 * kPieceBytes);
          for (int i = 0; i < 2; ++i)
            tma_load_3d(staging + i * kPieceBytes, &maps.in[i], &inbar[turn], 0, static_cast<int32_t>(row0) + r,
                        col0 / 64, policy_evict_first());
        }
        ++asked;
      };
      // A warp whose wait gave up leaves its turn only by a vote, and a vote comes
      // before any other barrier of the turn: its four warps have the tile, or all go.
      const bool early = kMode == kDownBwd && turn * 32 < rows;
      if constexpr (kMode == kDownBwd) {  // before the accumulator is waited for
        if (leader) tma_store_wait_read<0>();
        __syncwarp();
        if (vote_any(!ok, turn)) break;  // (as a barrier, what staging_free has)
        if (early) ask(turn * 32);
      }
      if (real && c.k > 0) ok = mbar_wait(&tfull[a], (tcount >> 1) & 1u, abort_flag, status);
      if (vote_any(!ok, turn)) {
        if (early) {
          int no_abort = 0;
          mbar_wait(&inbar[turn], (asked - 1) & 1u, &no_abort, status);
        }
        break;
      }
      if (c.last) break;
      if (lane == 0) ring_release(ring, n, rank, rempty0);
      if (!c.ok) continue;
      tc_fence_after();
      if (c.k > 0) ++tcount;
      // the accumulator has been read (by this warp)
      auto release = [&]() {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_peer(tempty0 + 8u * a);
      };
      if constexpr (kMode == kDownBwd) {
        // pieces of 32 rows, the turns' in turn
        if (!early) release();
        bool stop = false;
        for (int r = turn * 32; r < rows; r += kTurns * 32) {
          uint32_t v[32];
          load_piece(tb + a * kTileN + r, v);
          tmem_ld_wait();
          if (r + kTurns * 32 >= rows) release();
          // (where the wait gives up, the values are not used)
          const bool there = mbar_wait(&inbar[turn], (asked - 1) & 1u, abort_flag, status);
          const uint32_t at = smem_u32(staging) + staged_at(lane & 7, 4 * q + (lane >> 3), 32);
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
          fence_proxy_async_smem();
          if (vote_any(!there, turn)) {
            int no_abort = 0;
            mbar_wait(&inbar[turn], (asked - 1) & 1u, &no_abort, status);
            stop = true;
            break;
          }
          leave(staging, out.d[0], &maps.out[0], r, 32);
          leave(staging + kPieceBytes, out.d[1], &maps.out[1], r, 32);
          if (leader) tma_store_commit();
          if (r + kTurns * 32 < rows) {
            staging_free();
            ask(r + kTurns * 32);
          }
        }
        if (stop) break;
      } else {
        // a turn's 128 rows: all rounded to registers, the accumulator released,
        // then staged and stored HEIGHT rows at a time
        const int first = turn * (kTileN / kTurns);
        uint32_t packed[4][16];
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          if ((kMode != kWeightBwd || c.k > 0) && first + 32 * i < rows) {
            uint32_t v[2][32];
            load_piece(tb + a * kTileN + first + 32 * i, v[0]);
            load_piece(tb + a * kTileN + first + 32 * i + 32, v[1]);  // (in TMEM whatever the rows)
            tmem_ld_wait();
            round_piece(v[0], packed[i]);
            round_piece(v[1], packed[i + 1]);
          } else {  // an expert without rows: its gradient is zero
#pragma unroll
            for (int j = 0; j < 16; ++j) packed[i][j] = packed[i + 1][j] = 0u;
          }
        }
        if (c.k > 0) release();
#pragma unroll
        for (int i = 0; i < 4; i += C::HEIGHT / 32) {
          const int r = first + 32 * i;
          uint8_t* buf = staging + (C::BUFS > 1 ? i / (C::HEIGHT / 32) * C::HEIGHT * 256 : 0);
          if (r < rows) {
            if (leader) tma_store_wait_read<C::BUFS - 1>();
            __syncwarp();
            named_barrier_sync(3 + turn, 128);
#pragma unroll
            for (int j = 0; j < C::HEIGHT / 32; ++j)
              if (r + 32 * j < rows)
                stage_piece(smem_u32(buf) + j * 32 * 128, q, packed[i + j], lane, C::HEIGHT);
            fence_proxy_async_smem();
            named_barrier_sync(3 + turn, 128);
            const int mat = kMode == kWeightBwd ? c.mat : 0;
            leave(buf, out.d[mat], &maps.out[mat], r, C::HEIGHT);
          }
          if (leader) tma_store_commit();  // (a group for each buffer, of nothing where r lies behind the rows)
        }
      }
    }
    if (leader) tma_store_wait_all<0>();  // this thread's stores are written
    __syncwarp();
  } else if (warp == kSchedWarp) {
    if (rank == 0)
      schedule<kMode>(ring, p, off_pad, counts, blockIdx.x >> 1, gridDim.x >> 1, lane, abort_flag, status, sched);
    __syncwarp();
  } else if constexpr (kMode == kWeightBwd) {
    // ---------------------------------------------------------- clearing (both CTAs)
    uint32_t it = 0, bit = 0;
    uint32_t phases = 0;  // bit s: parity of the next use of stage s's barriers
    for (uint32_t n = 0;; ++n) {
      Tile c{};
      const bool got = ring_get(ring, n, rank, c, abort_flag, status);
      if (__any_sync(0xffffffffu, !got) || c.last) break;
      if (lane == 0) ring_release(ring, n, rank, rempty0);
      if (!c.ok) continue;
      it += stages_of(c.k);
      if (c.load_b) bit += stages_of(c.k);
      if (!has_tail(c)) continue;
      const uint32_t s = (it - 1) % C::STAGES;
      const uint32_t ph = (phases >> s) & 1u;
      phases ^= 1u << s;
      if (__any_sync(0xffffffffu, !mbar_wait(&tail[s], ph, abort_flag, status))) break;
      const int first = c.k & (kStageK - 1), last = (first + 15) & ~15;
      // lane: box (two of each operand, or one of the second) and 16-byte chunk
      const int slot = lane < 16 ? static_cast<int>(s) : C::STAGES + static_cast<int>((bit - 1) % C::STAGES);
      uint8_t* box = smem + slot * kOperandBytes + ((lane >> 3) & 1) * kBoxBytes + (lane & 7) * 16;
      if (lane < 16 || c.load_b)
        for (int r = first; r < last; ++r) *reinterpret_cast<uint4*>(box + r * 128) = make_uint4(0u, 0u, 0u, 0u);
      fence_proxy_async_smem();
      __syncwarp();
      bool ok = true;
      if (lane == 0) {
        if (rank == 0) {
          ok = mbar_wait<true>(&cleared[s], ph, abort_flag, status);
          if (ok) mbar_arrive(&full[s]);
        } else {
          mbar_arrive_peer(map_to_cta(&cleared[s], 0));
        }
      }
      if (__any_sync(0xffffffffu, !ok)) break;
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
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

template <int kMode>
cudaError_t launch(const moe_shape& s, const TrainMaps& m, const TrainOut& out, const int32_t* off_pad,
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
      err = cudaFuncSetAttribute(train_gemm_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
      if (err != cudaSuccess) return err;
      if (dev < 64) done[dev] = true;
    }
  }
  const int64_t ti = (s.I + 255) / 256, th = (s.H + 255) / 256;
  int64_t clusters = num_sms / 2;
  if (clusters > kMaxDrawers) clusters = kMaxDrawers;
  // Windows of 256 rows, or of 128 or 64 as long as every tile has a cluster of its
  // own: a tile then loads its weights for fewer rows, but takes less time (one
  // expert of 3968 x 1408, 500 rows: down 31 us with 256 rows, 19 with 64; where 64
  // would give more tiles than clusters, up 21 us with 256 and 29 with 64).
  const int64_t R = static_cast<int64_t>(s.T) * s.k, touched = s.E < R ? s.E : R;
  const int64_t cols = kMode == kDownBwd ? ti : th;
  int window = kTileN;
  while (window > 64 && (R / (window / 2) + touched) * cols <= clusters) window /= 2;
  // One expert has all rows, and its windows are taken as they fill the last wave of
  // tiles best, a tile costing its rows and half a tile's more (5003 rows, 2176 x 5760:
  // up 164 us with 256 rows, 154 so; 3000 rows, 2048 x 2048: down 44 and 35, up 61 and
  // 45; without the constant, 16384 rows of 4096 x 4096: down 474 where 256 rows take
  // 376).
  if (s.E == 1 && window == kTileN) {
    int64_t best = 0;
    for (int w = kTileN; w >= kTileN / 2; w -= 16) {
      const int64_t cost = ((R + w - 1) / w * cols + clusters - 1) / clusters * (w + kTileN / 2);
      if (best == 0 || cost < best) {
        best = cost;
        window = w;
      }
    }
  }
  const int64_t tiles = kMode == kWeightBwd ? s.E * 3 * ti * th : (R / window + touched) * cols;
  // tiles handed out ahead: enough that the loads of eight stages know theirs
  // (what a cluster has been handed no other can take)
  const int64_t k = kMode == kDownBwd ? s.H : kMode == kUpBwd ? 2 * s.I : static_cast<int64_t>(s.T) * s.k / s.E;
  const int64_t stages = k / kStageK + 1;
  int64_t ahead = 3 + 8 / stages;
  if (ahead > kTileRing) ahead = kTileRing;
  // Runs of at most three tiles, and at least sixteen of them for every cluster (64
  // experts of 4096 x 1536, 256 rows each on average: 555 us with runs of one tile, 521
  // with three, 528 with six, 538 with eight; 320 rows 640, 585, 580, 592; 16 rows,
  // which load little, 383, 385, 391, 393).
  int64_t run = tiles / (16 * clusters);
  run = run < 1 ? 1 : run > 3 ? 3 : run;
  auto even = [run](int64_t n) {  // length of n tiles' runs, as even as they come
    const int64_t runs = (n + run - 1) / run;
    return (n + runs - 1) / runs;
  };
  Problem p = {s.E, s.H, s.I, window, 0, 0, 0, 0, static_cast<uint32_t>(ahead), max_rows_of(s)};
  p.len_x = static_cast<int>(even(2 * ti));
  p.len_h = static_cast<int>(even(th));
  p.runs_x = static_cast<int>((2 * ti + p.len_x - 1) / p.len_x);
  p.runs_h = static_cast<int>((th + p.len_h - 1) / p.len_h);
  if (tiles < clusters) clusters = tiles;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * clusters));
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
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
  return cudaLaunchKernelEx(&cfg, train_gemm_kernel<kMode>, m, out, off_pad, counts,
                            p, status, sched);
}

}  // namespace

cudaError_t launch_down_backward(const moe_shape& s, const TrainMaps& m, const TrainOut& out, const int32_t* off_pad,
                                 const int32_t* counts, uint32_t* status, uint32_t* sched, int num_sms,
                                 cudaStream_t st) {
  return launch<kDownBwd>(s, m, out, off_pad, counts, status, sched, num_sms, st);
}

cudaError_t launch_up_backward(const moe_shape& s, const TrainMaps& m, const TrainOut& out, const int32_t* off_pad,
                               const int32_t* counts, uint32_t* status, uint32_t* sched, int num_sms,
                               cudaStream_t st) {
  return launch<kUpBwd>(s, m, out, off_pad, counts, status, sched, num_sms, st);
}

cudaError_t launch_weight_backward(const moe_shape& s, const TrainMaps& m, const TrainOut& out, const int32_t* off_pad,
                                   const int32_t* counts, uint32_t* status, uint32_t* sched, int num_sms,
                                   cudaStream_t st) {
  return launch<kWeightBwd>(s, m, out, off_pad, counts, status, sched, num_sms, st);
}

}  // namespace moe
