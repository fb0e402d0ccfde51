// moe_combine_backward.cu -- gradients of the weighted combine and of the
// routing weights.
//
// With out[t] = sum_j w[t, j] Y[row(t, j)] and w[t, :] the softmax of token t's
// picked logits (what softmax over all, top-k and renormalisation come to):
//   dY[row(t, j)] = w[t, j] dout[t]
//   dw[t, j]      = <dout[t], Y[row(t, j)]>
//   dlogits[t, e] = sum over picks j with id e of w[t, j] (dw[t, j] - sum_l w[t, l] dw[t, l])
// One pass: every row of Y is read once and the same row of dY written once, which
// is what bounds it (dout is read once): 16384 tokens of 4096 columns, 8 picks, 2.29
// GB in 343 us, 0.98 of the measured copy rate.
//
// A token is taken by one warp, or by the 2, 4 or 8 warps of a group where tokens
// are fewer than resident warps; each lane keeps 8 columns of dout and of every
// pick's row at a time, and its part of the k products in float32.  The group's
// parts meet in shared memory in a fixed order: no atomics.
// Inputs may be what an earlier kernel of the chain wrote: read past L1 (__ldcg).
#include <cstdint>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWarps = 8;

// two bf16 of `y` times those of `d`, added to acc in order
__device__ __forceinline__ float dot2(uint32_t y, uint32_t d, float acc) {
  acc = fmaf(bf16lo_to_f32(y), bf16lo_to_f32(d), acc);
  return fmaf(bf16hi_to_f32(y), bf16hi_to_f32(d), acc);
}
__device__ __forceinline__ uint32_t scale2(uint32_t d, float w) {
  return pack_bf16x2(w * bf16lo_to_f32(d), w * bf16hi_to_f32(d));
}

template <int KMAX>
__global__ void __launch_bounds__(kWarps * 32) combine_backward_kernel(
    const uint16_t* __restrict__ Y, const int32_t* __restrict__ scatter_idx, const int32_t* __restrict__ topk_ids,
    const float* __restrict__ topk_w, const uint16_t* __restrict__ dout, int T, int H, int E, int k, int64_t max_rows,
    int group, uint16_t* __restrict__ dY, float* __restrict__ dlogits, uint32_t* __restrict__ status) {
  __shared__ float s_part[kWarps][KMAX];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int part = warp & (group - 1);  // this warp's place in its token's group (group = 1, 2, 4 or 8)
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kWarps / group) + warp / group;
  const bool there = t < T;
  pdl_wait();
  int my_row = -1, my_id = -1;
  float my_w = 0.0f;
  if (there && lane < k) {
    const int64_t r = __ldcg(scatter_idx + t * k + lane);
    my_w = __ldcg(topk_w + t * k + lane);
    my_id = __ldcg(topk_ids + t * k + lane);
    if (r >= 0 && r < max_rows) my_row = static_cast<int>(r);
    if (part == 0 && (my_row < 0 || my_id < 0 || my_id >= E)) record_status(status, kStatusBounds);
  }
  int rows[KMAX];
  float w[KMAX], acc[KMAX];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    rows[j] = __shfl_sync(0xffffffffu, my_row, j);
    w[j] = __shfl_sync(0xffffffffu, my_w, j);
    acc[j] = 0.0f;
  }
  if (there) {
    const int vpr = H / 8;  // 16-byte vectors per row
    const uint4* d4 = reinterpret_cast<const uint4*>(dout) + t * vpr;
    const uint4* y4 = reinterpret_cast<const uint4*>(Y);
    uint4* o4 = reinterpret_cast<uint4*>(dY);
    for (int v = part * 32 + lane; v < vpr; v += group * 32) {
      const uint4 d = __ldcg(d4 + v);
      uint4 y[KMAX];
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        y[j] = make_uint4(0u, 0u, 0u, 0u);
        if (j < k && rows[j] >= 0) y[j] = __ldcg(y4 + static_cast<int64_t>(rows[j]) * vpr + v);
      }
#pragma unroll
      for (int j = 0; j < KMAX; ++j) {
        if (j < k && rows[j] >= 0) {
          acc[j] = dot2(y[j].w, d.w, dot2(y[j].z, d.z, dot2(y[j].y, d.y, dot2(y[j].x, d.x, acc[j]))));
          o4[static_cast<int64_t>(rows[j]) * vpr + v] =
              make_uint4(scale2(d.x, w[j]), scale2(d.y, w[j]), scale2(d.z, w[j]), scale2(d.w, w[j]));
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    if (lane == 0) s_part[warp][j] = acc[j];
  }
  if (group == 1) __syncwarp();
  else __syncthreads();
  if (!there) return;
  // lane j: the gradient of pick j's logit
  float dw = 0.0f;
  if (lane < k)
    for (int i = 0; i < group; ++i) dw += s_part[warp - part + i][lane];
  float mean = 0.0f;
  for (int j = 0; j < k; ++j) mean += __shfl_sync(0xffffffffu, my_w * dw, j);
  const float dl = my_w * (dw - mean);
  // the group's warps write the token's row of dlogits
  for (int e0 = part * 32; e0 < E; e0 += group * 32) {
    const int e = e0 + lane;
    float v = 0.0f;
    for (int j = 0; j < k; ++j) {
      const float d = __shfl_sync(0xffffffffu, dl, j);
      if (__shfl_sync(0xffffffffu, my_id, j) == e) v += d;
    }
    if (e < E) dlogits[t * E + e] = v;
  }
}

}  // namespace

cudaError_t launch_combine_backward(const moe_shape& s, const uint16_t* Y, const int32_t* scatter_idx,
                                    const int32_t* topk_ids, const float* topk_w, const uint16_t* dout, uint16_t* dY,
                                    float* dlogits, uint32_t* status, int num_sms, cudaStream_t st) {
  // warps per token: as many as fill 16 warps per SM, at most one per 256 columns
  int group = 1;
  while (group < kWarps && static_cast<int64_t>(s.T) * group < static_cast<int64_t>(num_sms) * 16 &&
         s.H >= 512 * group)
    group *= 2;
  const int per = kWarps / group;
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(s.T) + per - 1) / per));
  if (s.k <= 8)
    return launch_pdl(combine_backward_kernel<8>, grid, dim3(kWarps * 32), 0, st, Y, scatter_idx, topk_ids, topk_w,
                      dout, s.T, s.H, s.E, s.k, max_rows_of(s), group, dY, dlogits, status);
  return launch_pdl(combine_backward_kernel<16>, grid, dim3(kWarps * 32), 0, st, Y, scatter_idx, topk_ids, topk_w,
                    dout, s.T, s.H, s.E, s.k, max_rows_of(s), group, dY, dlogits, status);
}

}  // namespace moe
