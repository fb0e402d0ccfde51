// moe_int8_rows.cu -- the grouped products on 8-bit integers for a few rows (the
// decoding of single tokens), from integer dot products: the same bits as
// moe_int8_gemm.cu gives while every sum and partial sum is below 2^24 (always for a
// reduction of up to 1024).  Beyond that the sums here are still exact and rounded
// once, where float32 sums round on the way.
//
// With one row per expert the product is a stream of weight rows against one
// vector each: 100 MB of gate and up codes for a token of 8 experts of 4096 x 1536,
// 15 us at the copy rate, and only 48 tiles for the tensor cores' 76 clusters.  Here
// a warp takes two weight rows at a time (gate and up of one column, or two
// neighbouring columns of down), its lanes 16 codes each per load, eight loads on
// their way, and adds products of four with dp4a; the rows come through L1, which
// the warps of an SM share.  The sums are 32-bit integers: exact.
#include <cstdint>

#include "moe_device.cuh"
#include "moe_epilogue.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMaxExperts = 256;
constexpr int kWarps = 8;
constexpr int kRows = 4;   // rows of an expert at a time (more read the weights again, from L2)
constexpr int kLoads = 4;  // loads of 512 bytes per weight row on their way

template <bool kUp>
__global__ void __launch_bounds__(kWarps * 32) int8_rows_kernel(
    const int8_t* __restrict__ x, const float* __restrict__ sx, const int8_t* __restrict__ w0,
    const float* __restrict__ s0, const int8_t* __restrict__ w1, const float* __restrict__ s1,
    const int32_t* __restrict__ off_pad, const int32_t* __restrict__ counts, int E, int K, int N, int64_t max_rows,
    uint16_t* __restrict__ D, uint32_t* __restrict__ status) {
  __shared__ int s_expert[kMaxExperts], s_first[kMaxExperts], s_count[kMaxExperts];  // those with rows
  __shared__ int s_base[kWarps + 1];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  pdl_wait();
  {  // a thread per expert: the ones with rows, in order
    const int e = threadIdx.x;
    int c = 0;
    int64_t first = 0;
    if (e < E) {
      c = __ldcg(counts + e);
      first = __ldcg(off_pad + e);
      const int64_t end = __ldcg(off_pad + e + 1);
      // an expert whose rows do not lie inside its 128-row blocks and the buffers has none
      if (c < 0 || first < 0 || (first & 127) != 0 || (end & 127) != 0 || first + c > end || end > max_rows) {
        if (blockIdx.x == 0) record_status(status, kStatusBounds);
        c = 0;
      }
    }
    const uint32_t has = __ballot_sync(0xffffffffu, c > 0);
    if (lane == 0) s_base[warp + 1] = __popc(has);
    if (threadIdx.x == 0) s_base[0] = 0;
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = 0; i < kWarps; ++i) s_base[i + 1] += s_base[i];
    __syncthreads();
    if (c > 0) {
      const int at = s_base[warp] + __popc(has & ((1u << lane) - 1u));
      s_expert[at] = e;
      s_first[at] = static_cast<int>(first);
      s_count[at] = c;
    }
    __syncthreads();
  }
  const int per = kUp ? N : N / 2;  // items of an expert
  const int64_t items = static_cast<int64_t>(s_base[kWarps]) * per;
  const int vecs = K / 16;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items;
       item += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int at = static_cast<int>(item / per);
    const int i = static_cast<int>(item - static_cast<int64_t>(at) * per);
    const int64_t n0 = static_cast<int64_t>(s_expert[at]) * N + (kUp ? i : 2 * i);
    const int64_t n1 = kUp ? n0 : n0 + 1;
    const uint4* a = reinterpret_cast<const uint4*>(w0 + n0 * K) + lane;
    const uint4* b = reinterpret_cast<const uint4*>((kUp ? w1 : w0) + n1 * K) + lane;
    const float sa = __ldcg(s0 + n0), sb = __ldcg((kUp ? s1 : s0) + n1);
    for (int r0 = 0; r0 < s_count[at]; r0 += kRows) {
      const int rows = min(kRows, s_count[at] - r0);  // alike for the warp
      const int64_t row = s_first[at] + r0;
      const uint4* xr = reinterpret_cast<const uint4*>(x + row * K) + lane;
      int acc[kRows][2] = {};
      for (int v0 = 0; v0 < vecs; v0 += 32 * kLoads) {
        uint4 p[kLoads], q[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          p[u] = q[u] = make_uint4(0u, 0u, 0u, 0u);
          if (v0 + 32 * u + lane < vecs) {
            p[u] = __ldcg(a + v0 + 32 * u);
            q[u] = __ldcg(b + v0 + 32 * u);
          }
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
          if (r < rows) {
#pragma unroll
            for (int u = 0; u < kLoads; ++u) {
              if (v0 + 32 * u + lane < vecs) {
                const uint4 c = __ldca(xr + static_cast<int64_t>(r) * vecs + v0 + 32 * u);
                const int xs[4] = {static_cast<int>(c.x), static_cast<int>(c.y), static_cast<int>(c.z),
                                   static_cast<int>(c.w)};
                const int ps[4] = {static_cast<int>(p[u].x), static_cast<int>(p[u].y), static_cast<int>(p[u].z),
                                   static_cast<int>(p[u].w)};
                const int qs[4] = {static_cast<int>(q[u].x), static_cast<int>(q[u].y), static_cast<int>(q[u].z),
                                   static_cast<int>(q[u].w)};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  acc[r][0] = __dp4a(xs[j], ps[j], acc[r][0]);
                  acc[r][1] = __dp4a(xs[j], qs[j], acc[r][1]);
                }
              }
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r < rows) {
          const int g = __reduce_add_sync(0xffffffffu, acc[r][0]);
          const int u = __reduce_add_sync(0xffffffffu, acc[r][1]);
          if (lane == r) {
            const float s = __ldcg(sx + row + r);
            const float y0 = static_cast<float>(g) * s * sa, y1 = static_cast<float>(u) * s * sb;
            if (kUp)
              D[(row + r) * N + i] = static_cast<uint16_t>(pack_bf16x2(silu_mul(y0, y1), 0.0f));
            else
              *reinterpret_cast<uint32_t*>(D + (row + r) * N + 2 * i) = pack_bf16x2(y0, y1);
          }
        }
      }
    }
  }
}

template <bool kUp>
cudaError_t launch(const moe_shape& s, const int8_t* x, const float* sx, const int8_t* w0, const float* s0,
                   const int8_t* w1, const float* s1, uint16_t* D, const int32_t* off_pad, const int32_t* counts,
                   uint32_t* status, int num_sms, cudaStream_t st) {
  const int K = kUp ? s.H : s.I, N = kUp ? s.I : s.H;
  const int64_t R = static_cast<int64_t>(s.T) * s.k;
  const int64_t items = (R < s.E ? R : s.E) * (kUp ? N : N / 2);
  int64_t blocks = (items + kWarps - 1) / kWarps;
  if (blocks > 3 * num_sms) blocks = 3 * num_sms;
  return launch_pdl(int8_rows_kernel<kUp>, dim3(static_cast<unsigned>(blocks)), dim3(kWarps * 32), 0, st, x, sx, w0,
                    s0, w1, s1, off_pad, counts, s.E, K, N, max_rows_of(s), D, status);
}

}  // namespace

// Up to two tokens, or half a row per expert on average, but at most 24 rows in all,
// and 8 tokens, so that the longest expert's weights are read twice at most.  From
// memory (behind a 256 MB fill), us, this way and on the tensor cores, gate/up | down (a rule on the rows
// serves both, as their limits are near to one another):
//   4096 x 1536, 64 experts, 8 per token: 8 rows 36 | 23 and 33 | 23 (18 | 10 and 28 |
//     17 where the weights lie in L2), 16 rows 56 | 38 and 79 | 42, 24 rows 70 | 48 and
//     79 | 42, 32 rows 85 | 58 and 81 | 44
//   2048 x 768, 128 experts, 8 per token: 8 rows 16 | 14 and 23 | 19, 16 rows 24 | 19
//     and 25 | 19, 24 rows 29 | 23 and 27 | 29 (13 | 13 and 20 | 22 in L2), 32 rows
//     38 | 27 and 48 | 29, 64 rows 58 | 44 and 48 | 30
//   7168 x 2048, 256 experts, 8 per token: 8 rows 64 | 38 and 56 | 50, 16 rows 107 | 60
//     and 128 | 54, 24 rows 150 | 83 and 132 | 76, 128 rows 609 | 330 and 480 | 240
//   2048 x 1024, 256 experts, 1 per token: 4 rows 15 | 11 and 23 | 19; 8 rows 19 | 15
//     and 25 | 19, all in one expert 23 | 16 and 23 | 19; 16 rows 27 | 19 and 27 | 23,
//     in one expert 36 | 25 and 23 | 19; 128 rows 117 | 79 and 89 | 54, in one expert
//     230 | 138 and 25 | 21
bool int8_few_rows(const moe_shape& s) {
  const int64_t rows = static_cast<int64_t>(s.T) * s.k;
  return rows <= 24 && s.T <= 2 * kRows && (s.T <= 2 || 2 * rows <= s.E);
}

cudaError_t launch_int8_up_rows(const moe_shape& s, const int8_t* x, const float* x_scales, const int8_t* wg,
                                const float* wg_scales, const int8_t* wu, const float* wu_scales, uint16_t* h,
                                const int32_t* off_pad, const int32_t* counts, uint32_t* status, int num_sms,
                                cudaStream_t st) {
  return launch<true>(s, x, x_scales, wg, wg_scales, wu, wu_scales, h, off_pad, counts, status, num_sms, st);
}

cudaError_t launch_int8_down_rows(const moe_shape& s, const int8_t* h, const float* h_scales, const int8_t* wd,
                                  const float* wd_scales, uint16_t* Y, const int32_t* off_pad, const int32_t* counts,
                                  uint32_t* status, int num_sms, cudaStream_t st) {
  return launch<false>(s, h, h_scales, wd, wd_scales, wd, wd_scales, Y, off_pad, counts, status, num_sms, st);
}

}  // namespace moe
