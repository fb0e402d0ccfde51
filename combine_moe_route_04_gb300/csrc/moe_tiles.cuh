// moe_tiles.cuh -- tiles of the grouped products whose CTAs work alone: windows of
// an expert's rows, the tile counter, the ring that hands tile indices to a CTA's
// roles, and the activation.
#pragma once

#include <cstdint>

#include "moe_device.cuh"

namespace moe {

constexpr int kMaxExperts = 256;
constexpr int kTileRing = 4;  // tile indices on their way from the producer

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
// launch.  That CTA also knows whether the launch started from a cleared
// counter: the word behind it counts the CTAs that have stopped (bits 0-9),
// sums their indexes plus one (bits 10-29), and gets bit 30 from the one that
// drew 0, the first value of a cleared counter.  With anything else in either
// word the sum comes out wrong (tiles may have been left out): an error.
constexpr int kMaxGrid = 1023;
__device__ __forceinline__ uint32_t stopped(uint32_t ctas, uint32_t index_sum, bool drew_zero) {
  return ctas | (index_sum << 10) | (drew_zero ? 1u << 30 : 0u);
}
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

// silu(g) * u with the sigmoid on the SFU.  The exponent g log2 e is rounded
// before ex2, so below zero the relative error grows with |g|, to about
// |g| 2^-24 and a few ulps (2^-17 at g = -88, below which the result is the
// limit 0, as in the bf16 GEMM): far under h's rounding to bf16, 2^-9.
__device__ __forceinline__ float silu_mul(float g, float u) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return g * r * u;
}

}  // namespace moe
