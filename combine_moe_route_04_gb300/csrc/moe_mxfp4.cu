// moe_mxfp4.cu -- quantisation to MXFP4 and back.
//
// A block of 32 consecutive elements x of a row gets the scale byte
//   s = clamp(floor(log2(max|x|)) - 2 + 127, 0, 254)
// and the codes e2m1(x 2^(127 - s)), rounded to nearest even and saturated at
// 6 (the OCP microscaling rule).  Every step is exact in float32 but the
// rounding to e2m1 itself, so the results are those of the definition to the
// bit.  All four kernels move data once and are bound by memory: 16384 x 4096
// rows take 25.6 us (6.65 TB/s), 64 weights of 4096 x 1536 145 us (7.0 TB/s) and
// 149 us back (6.85 TB/s); the measured copy rate is 6.7 TB/s.  On the way the
// rows' kernel was bound by instructions (38.9 us with 64-bit divisions and
// maxima one bf16 at a time), hence the two-dimensional grid, the 16-bit pair
// maxima and the products by the scale in pairs of bf16.
// Inputs may be what an earlier kernel of a chain of dependent launches wrote, so
// they are read past L1 (__ldcg), not through the non-coherent path.
#include <cstdint>

#include "moe_internal.h"
#include "moe_mxfp4.cuh"

namespace moe {
namespace {

constexpr int kSegCols = 1024;  // columns per work item: 4 x (32 lanes x 8 elements)

// One warp per (row, 1024-column segment; blockIdx.y): a lane holds 8 elements
// (16 bytes in, 4 bytes of codes out), four lanes a block, sixteen lanes the
// four blocks of a scale word.  Rows past the last one, up to a multiple of
// 128, get zero scales so that a tile of scales is always written whole.
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int64_t cols,
                                                            uint8_t* __restrict__ codes,
                                                            uint8_t* __restrict__ scales) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kSegCols + lane * 8;
  const int left = static_cast<int>(cols - c0);  // a lane's piece u is there when 256 u < left
  const uint16_t* src = x + r * cols + c0;
  uint8_t* dst = codes + (r * cols + c0) / 2;
  uint8_t* sc = scales + scale_word_offset(r, c0 / 128, cols / 128);
  const bool there = r < rows;
  pdl_wait();
  uint4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (there && u * 256 < left) v[u] = __ldcg(reinterpret_cast<const uint4*>(src + u * 256));
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t s = block_scale_of_quad(v[u]);
    const uint32_t w = scale_word_of_half(s, lane);
    if (u * 256 < left) {  // alike for the sixteen lanes of a scale word
      if (there) *reinterpret_cast<uint32_t*>(dst + u * 128) = quantize_bf16x8(v[u], s);
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(sc + u * 1024) = w;
    }
  }
}

// The inverse, same work split: 4 bytes of codes and the scale byte in, eight
// bf16 out (every MXFP4 value but those past bf16's range is a bf16).
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const uint8_t* __restrict__ codes,
                                                              const uint8_t* __restrict__ scales, int64_t rows,
                                                              int64_t cols, uint16_t* __restrict__ x) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int64_t c0 = static_cast<int64_t>(blockIdx.y) * kSegCols + lane * 8;
  const int left = static_cast<int>(cols - c0);
  const uint8_t* src = codes + (r * cols + c0) / 2;
  const uint8_t* sc = scales + scale_word_offset(r, c0 / 128, cols / 128) + ((lane >> 2) & 3);
  uint16_t* dst = x + r * cols + c0;
  if (r >= rows) return;
  pdl_wait();
  uint32_t code[4], sb[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    code[u] = sb[u] = 0u;
    if (u * 256 < left) {
      code[u] = __ldcg(reinterpret_cast<const uint32_t*>(src + u * 128));
      sb[u] = __ldcg(sc + u * 1024);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t m = scale_bf16(sb[u]) * 0x10001u;
    uint4 o;
    dequantize_bf16x4(code[u], m, o.x, o.y);
    dequantize_bf16x4(code[u] >> 16, m, o.z, o.w);
    if (u * 256 < left) *reinterpret_cast<uint4*>(dst + u * 256) = o;
  }
}

// Weights w [E][K][N] to codes [E][N][K/2]: the reduction axis K becomes the
// contiguous one.  A CTA takes 64 columns n and 256 k: warp b holds the block
// of 32 k's, a lane two neighbouring columns (32 loads of 4 bytes, 128
// contiguous bytes per warp), so a block's maximum and its 16 code bytes form
// in one thread; the codes cross shared memory once so that each column's 128
// bytes leave together.
constexpr int kWn = 64, kWk = 256;
constexpr int kCodePitch = 128 + 16;  // bytes per column in shared memory (16-byte accesses, padded)

__global__ void __launch_bounds__(256) quantize_weights_kernel(const uint16_t* __restrict__ w, int64_t K, int64_t N,
                                                               uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales) {
  __shared__ __align__(16) uint8_t s_code[kWn * kCodePitch];
  __shared__ __align__(4) uint8_t s_scale[kWn * 8];
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int b = threadIdx.x >> 5;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kWn;
  const int64_t k0 = static_cast<int64_t>(blockIdx.y) * kWk;
  const int64_t e = blockIdx.z;
  const int blocks = static_cast<int>(min(static_cast<int64_t>(8), (K - k0) / 32));
  if (b < blocks) {
    const uint16_t* src = w + (e * K + k0 + 32 * b) * N + n0 + 2 * lane;
    uint32_t v[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __ldcg(reinterpret_cast<const uint32_t*>(src + i * N));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < 32; ++i) m = max(m, (v[i] >> (16 * h)) & 0x7FFFu);
      const uint32_t s = scale_byte(m);
      const float inv = s == kScaleNan ? 0.0f : scale_inverse(s);
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float f[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          f[i] = (h == 0 ? bf16lo_to_f32(v[8 * q + i]) : bf16hi_to_f32(v[8 * q + i])) * inv;
        o[q] = s == kScaleNan ? 0u : pack_e2m1x8(f);
      }
      const int n = 2 * lane + h;
      *reinterpret_cast<uint4*>(s_code + n * kCodePitch + b * 16) = make_uint4(o[0], o[1], o[2], o[3]);
      s_scale[n * 8 + b] = static_cast<uint8_t>(s);
    }
  }
  __syncthreads();
  const int64_t row0 = e * N + n0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int n = static_cast<int>(threadIdx.x >> 3) + 32 * j;
    const int ch = threadIdx.x & 7;
    if (ch < blocks)
      *reinterpret_cast<uint4*>(codes + (row0 + n) * (K / 2) + k0 / 2 + ch * 16) =
          *reinterpret_cast<const uint4*>(s_code + n * kCodePitch + ch * 16);
  }
  if (threadIdx.x < 2 * kWn) {
    const int n = threadIdx.x >> 1, a = threadIdx.x & 1;
    if (4 * a < blocks)
      *reinterpret_cast<uint32_t*>(scales + scale_word_offset(row0 + n, k0 / 128 + a, K / 128)) =
          *reinterpret_cast<const uint32_t*>(s_scale + n * 8 + 4 * a);
  }
}

// Token rows quantised once and written to each of their k permuted rows: one
// warp per (token, 1024-column segment).
__global__ void __launch_bounds__(256) quantize_permute_kernel(const uint16_t* __restrict__ X,
                                                               const int32_t* __restrict__ scatter_idx, int T, int H,
                                                               int k, int64_t max_rows, uint8_t* __restrict__ codes,
                                                               uint8_t* __restrict__ scales,
                                                               uint32_t* __restrict__ status) {
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int c0 = static_cast<int>(blockIdx.y) * kSegCols + lane * 8;
  const int kb128 = H / 128;
  if (t >= T) return;  // a whole warp
  pdl_wait();
  int my_row = -1;  // lane j < k: row of (t, j)
  if (lane < k) {
    const int32_t r = __ldcg(scatter_idx + t * k + lane);
    if (r >= 0 && r < max_rows) my_row = r;
    else record_status(status, kStatusBounds);
  }
  uint4 v[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    v[u] = make_uint4(0u, 0u, 0u, 0u);
    if (c0 + u * 256 < H) v[u] = __ldcg(reinterpret_cast<const uint4*>(X + t * H + c0 + u * 256));
  }
  uint32_t code[4], word[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint32_t s = block_scale_of_quad(v[u]);
    word[u] = scale_word_of_half(s, lane);
    code[u] = quantize_bf16x8(v[u], s);
  }
  for (int j = 0; j < k; ++j) {
    const int64_t r = __shfl_sync(0xffffffffu, my_row, j);
    if (r < 0) continue;
    uint8_t* dst = codes + (r * H + c0) / 2;
    uint8_t* sc = scales + scale_word_offset(r, c0 / 128, kb128);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (c0 + u * 256 >= H) continue;
      *reinterpret_cast<uint32_t*>(dst + u * 128) = code[u];
      if ((lane & 15) == 0) *reinterpret_cast<uint32_t*>(sc + u * 1024) = word[u];
    }
  }
}

// one warp per row and segment, eight rows per CTA
dim3 grid_of(int64_t rows, int64_t cols) {
  return dim3(static_cast<unsigned>((rows + 7) / 8), static_cast<unsigned>((cols + kSegCols - 1) / kSegCols));
}

}  // namespace

cudaError_t launch_quantize_rows(const uint16_t* x, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                                 cudaStream_t st) {
  return launch_pdl(quantize_rows_kernel, grid_of((rows + 127) / 128 * 128, cols), dim3(256), 0, st, x, rows, cols,
                    codes, scales);
}

cudaError_t launch_dequantize_rows(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols,
                                   uint16_t* x, cudaStream_t st) {
  return launch_pdl(dequantize_rows_kernel, grid_of(rows, cols), dim3(256), 0, st, codes, scales, rows, cols, x);
}

cudaError_t launch_quantize_weights(const uint16_t* w, int E, int64_t K, int64_t N, uint8_t* codes, uint8_t* scales,
                                    cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(N / kWn), static_cast<unsigned>((K + kWk - 1) / kWk),
                  static_cast<unsigned>(E));
  return launch_pdl(quantize_weights_kernel, grid, dim3(256), 0, st, w, K, N, codes, scales);
}

cudaError_t launch_quantize_permute(const moe_shape& s, const uint16_t* X, const int32_t* scatter_idx, uint8_t* codes,
                                    uint8_t* scales, uint32_t* status, cudaStream_t st) {
  return launch_pdl(quantize_permute_kernel, grid_of(s.T, s.H), dim3(256), 0, st, X, scatter_idx, s.T, s.H, s.k,
                    max_rows_of(s), codes, scales, status);
}

}  // namespace moe
