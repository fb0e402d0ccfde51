// moe_int8.cu -- quantisation to 8-bit integers with one scale per row, and back.
//
// A row x gets the scale s = amax / 127 (float32, amax = max |x|) and the codes
//   q = 127 x / amax, rounded to the nearest integer, ties to even,
// and stands for q s.  The quotient is rounded as if it were exact: 127 x / amax
// of two bf16 values (8-bit significands) is either a tie n + 1/2 or at least
// 2^-17 of its power of two away from one, so it is formed as x * (127 / amax)
// (off by less than 2^-22), rounded to 19 bits behind the leading one, which
// restores a tie and crosses none, and then to an integer.
//
// The rows' kernel and the inverse move data once: 16384 x 4096 rows take 38 us (5.3
// TB/s; three quarters of the issue slots are used), their values 30.6 us (6.6 TB/s),
// the values of 64 weights of 4096 x 1536 171 us (7.1 TB/s).  The weights' kernel
// reads its columns once, up to 12288 rows of them, and longer ones twice.
// Inputs may be what an earlier kernel of a chain of dependent launches wrote, so
// they are read past L1 (__ldcg), not through the non-coherent path.
#include <cstdint>
#include <mutex>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr uint32_t kInfBits = 0x7F80u;  // bf16 magnitudes from here on are infinite or NaN

// the larger of the magnitudes of two pairs of bf16, per half
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, uint32_t v) { return __vmaxu2(m, v & 0x7FFF7FFFu); }
__device__ __forceinline__ uint32_t max_magnitude(uint32_t m, const uint4& v) {
  return max_magnitude(max_magnitude(max_magnitude(max_magnitude(m, v.x), v.y), v.z), v.w);
}

// Below 2^-64 and from 2^100, where 1 / amax may leave the normal numbers, x and
// amax are raised by this power of two first (exactly, but for elements that
// become subnormal, whose codes are 0 either way).
__device__ __forceinline__ float raise_of(uint32_t amax_bits) {
  return amax_bits < 0x1F80u ? 0x1p64f : amax_bits >= 0x7180u ? 0x1p-64f : 1.0f;
}
// 127 / (amax * raise), off by less than 2^-22; 0 for a row of zeros.
__device__ __forceinline__ float inverse_of(uint32_t amax_bits, float raise) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(__uint_as_float(amax_bits << 16) * raise));
  return amax_bits == 0u ? 0.0f : 127.0f * r;
}
// The scale amax / 127, NaN for a row that holds a NaN or an infinity.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
  return amax_bits >= kInfBits ? __uint_as_float(0x7FC00000u) : __fdiv_rn(__uint_as_float(amax_bits << 16), 127.0f);
}
// The code in the low byte: y rounded to 19 bits behind the leading one, then to an
// integer by adding 1.5 * 2^23 (the conversion instruction has an eighth of the
// adder's rate).
__device__ __forceinline__ uint32_t code_of(float y) {
  const float z = __uint_as_float((__float_as_uint(y) + 8u) & ~15u);
  return __float_as_uint(z + 12582912.0f);
}
__device__ __forceinline__ uint32_t pack4(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}
// Eight codes of v * raise * inv.
template <bool kRaise>
__device__ __forceinline__ uint2 codes8(const uint4& v, float raise, float inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = kRaise ? bf16lo_to_f32(w[i]) * raise : bf16lo_to_f32(w[i]);
    const float b = kRaise ? bf16hi_to_f32(w[i]) * raise : bf16hi_to_f32(w[i]);
    q[2 * i] = code_of(a * inv);
    q[2 * i + 1] = code_of(b * inv);
  }
  return make_uint2(pack4(q[0], q[1], q[2], q[3]), pack4(q[4], q[5], q[6], q[7]));
}

constexpr int kRowVecs = 4;  // 16-byte vectors of a row that a lane keeps

// Row t of x to row(s) of codes: row t itself, or (scatter_idx) the token's k
// permuted rows; with gather_idx, only rows of x that hold a token (x is then in
// expert order).  A row is taken by a group of 1, 2, 4 or 8 warps, enough to keep
// 8192 columns in registers between the maximum and the codes; further columns
// are read twice.
__global__ void __launch_bounds__(256, 5) quantize_rows_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                               const int32_t* __restrict__ scatter_idx, int k,
                                                               int64_t max_rows,
                                                               const int32_t* __restrict__ gather_idx,
                                                               const int32_t* __restrict__ num_blocks, int group,
                                                               int8_t* __restrict__ codes, float* __restrict__ scales,
                                                               uint32_t* __restrict__ status) {
  __shared__ uint32_t s_max[8];
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int warp = threadIdx.x >> 5;
  const int part = warp & (group - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (8 / group) + warp / group;
  pdl_wait();
  bool there = t < rows;
  if (there && gather_idx != nullptr)
    there = t < static_cast<int64_t>(__ldcg(num_blocks)) * kRowBlock && __ldcg(gather_idx + t) >= 0;
  const int vpr = cols / 8;
  const uint4* src = reinterpret_cast<const uint4*>(x) + t * vpr;
  const int step = group * 32;
  int c0 = part * 32 + lane;  // this lane's first vector
  uint4 v[kRowVecs];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (there && c0 + i * step < vpr) v[i] = __ldcg(src + c0 + i * step);
  }
  int64_t my_row = -1;  // lane j: the j-th row to write
  if (there && lane < k) {
    if (scatter_idx == nullptr) {
      my_row = t;
    } else {
      const int32_t r = __ldcg(scatter_idx + t * k + lane);
      if (r >= 0 && r < max_rows) my_row = r;
      else if (part == 0) record_status(status, kStatusBounds);
    }
  }
#pragma unroll
  for (int i = 0; i < kRowVecs; ++i) m = max_magnitude(m, v[i]);
  if (there)
    for (int c = c0 + kRowVecs * step; c < vpr; c += step) m = max_magnitude(m, __ldcg(src + c));
  m = max(m & 0xFFFFu, m >> 16);
  m = __reduce_max_sync(0xffffffffu, m);
  if (group > 1) {
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    m = 0u;
    for (int i = 0; i < group; ++i) m = max(m, s_max[warp - part + i]);
  }
  if (!there) return;
  const float raise = raise_of(m);
  const float inv = inverse_of(m, raise);
  if (part == 0 && my_row >= 0) scales[my_row] = scale_of(m);
  uint2* dst = reinterpret_cast<uint2*>(codes);
  for (;;) {
    uint2 q[kRowVecs];
    if (m >= kInfBits) {
#pragma unroll
      for (int i = 0; i < kRowVecs; ++i) q[i] = make_uint2(0u, 0u);
    } else if (raise == 1.0f) {
#pragma unroll
      for (int i = 0; i < kRowVecs; ++i) q[i] = codes8<false>(v[i], 1.0f, inv);
    } else {
#pragma unroll
      for (int i = 0; i < kRowVecs; ++i) q[i] = codes8<true>(v[i], raise, inv);
    }
    for (int j = 0; j < k; ++j) {
      const int64_t row = __shfl_sync(0xffffffffu, my_row, j);
      if (row < 0) continue;
      uint2* to = dst + row * vpr + c0;
#pragma unroll
      for (int i = 0; i < kRowVecs; ++i)
        if (c0 + i * step < vpr) to[i * step] = q[i];
    }
    c0 += kRowVecs * step;
    if (c0 - lane >= vpr) break;  // alike for the warp's lanes
#pragma unroll
    for (int i = 0; i < kRowVecs; ++i)
      if (c0 + i * step < vpr) v[i] = __ldcg(src + c0 + i * step);
  }
}

// Values bf16(q s): a thread takes kDeqVecs times 8 codes, a block's apart, so
// that a warp's stores are 512 contiguous bytes each.
constexpr int kDeqVecs = 4;
__global__ void __launch_bounds__(256) dequantize_rows_kernel(const int8_t* __restrict__ codes,
                                                              const float* __restrict__ scales, int64_t n8,
                                                              int vecs_per_row, uint16_t* __restrict__ x) {
  pdl_launch_dependents();
  pdl_wait();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (256 * kDeqVecs) + threadIdx.x;
  uint2 q[kDeqVecs];
  float s[kDeqVecs];
#pragma unroll
  for (int i = 0; i < kDeqVecs; ++i) {
    const int64_t v = first + 256 * i;
    if (v < n8) {
      q[i] = __ldcg(reinterpret_cast<const uint2*>(codes) + v);
      s[i] = __ldca(scales + v / vecs_per_row);
    }
  }
#pragma unroll
  for (int i = 0; i < kDeqVecs; ++i) {
    const int64_t v = first + 256 * i;
    if (v >= n8) return;
    const uint32_t w[2] = {q[i].x, q[i].y};
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t b = w[j >> 1] >> (16 * (j & 1));
      o[j] = pack_bf16x2(static_cast<float>(static_cast<int8_t>(b)) * s[i],
                         static_cast<float>(static_cast<int8_t>(b >> 8)) * s[i]);
    }
    reinterpret_cast<uint4*>(x)[v] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Weights w [E][K][N] to codes [E][N][K], the reduction axis K contiguous, and a
// scale per (e, n).  A cluster of kWCtas CTAs takes 32 columns of one expert, each CTA
// its share of their rows: a first pass over them (64 bytes each) for the maxima,
// which meet in distributed shared memory, a second one, in steps of kWk rows, for the
// codes, which cross shared memory once so that each column's bytes leave together.
// The first pass brings the rows to shared memory, each thread those that it takes in
// the second (kHeld; up to kMostHeld rows, two or three CTAs an SM, so that one's loads
// run under the others' arithmetic); longer columns are read twice, backwards the
// second time, when much of them is still in L2.
//
// 64 weights of 4096 x 1536 239 us with four CTAs of 1024 rows, where reading and
// writing once would take 178 (8 CTAs 276; two that read twice 275); of 1536 x 4096
// 230 with one (two 255, four 311; reading twice 255); of 2816 x 2048 237 with two (286);
// of 7168 x 2048 603 with eight (665); 7 of 1408 x 640, which fill no device, 8.2, 7.8
// and 7.0 with one, two and four.  So: as few CTAs as hold the rows, and more, up to
// four, where the grid leaves room.  (A cluster of eight that holds 64 columns in
// registers took 305 us for 4096 x 1536 and 436 for 1536 x 4096.)
constexpr int kWn = 32;
constexpr int kWeightThreads = 256;
constexpr int kWk = kWeightThreads / 4 * 4;  // four rows x eight columns per thread
constexpr int kMostHeld = 6 * kWk;           // rows of a CTA: 96 KB

template <int kWCtas, bool kHeld>
__global__ void __launch_bounds__(kWeightThreads, 4) quantize_weights_kernel(const uint16_t* __restrict__ w, int K,
                                                                             int N, int8_t* __restrict__ codes,
                                                                             float* __restrict__ scales) {
  __shared__ __align__(16) uint32_t s_codes[kWn * kWk / 4];
  __shared__ uint4 s_max[kWeightThreads / 32][4];
  __shared__ uint4 s_all[kWCtas][4];  // the CTAs' maxima
  if (kWCtas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_launch_dependents();
  pdl_wait();
  const uint32_t rank = kWCtas > 1 ? cluster_ctarank() : 0u;
  const int rows = K / kWCtas;  // a multiple of 16
  const int64_t first = static_cast<int64_t>(rank) * rows;
  const int cg = threadIdx.x & 3;   // columns 8 cg..
  const int kr = threadIdx.x >> 2;  // row of the thread, or group of four rows
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t e = blockIdx.z;
  const int64_t n0 = static_cast<int64_t>(blockIdx.x) * kWn;
  const uint4* src = reinterpret_cast<const uint4*>(w + (e * K + first) * N + n0) + cg;
  const int64_t pitch = N / 8;
  uint4 m = make_uint4(0u, 0u, 0u, 0u);
  extern __shared__ uint4 s_held[];
  auto more = [&](const uint4& v) {
    m.x = max_magnitude(m.x, v.x);
    m.y = max_magnitude(m.y, v.y);
    m.z = max_magnitude(m.z, v.z);
    m.w = max_magnitude(m.w, v.w);
  };
  if constexpr (kHeld) {  // each thread's own rows of the second pass
    uint4* to = s_held + threadIdx.x;
    for (int k = 4 * kr; k < rows; k += kWk, to += 4 * kWeightThreads)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + i * kWeightThreads)),
                     "l"(src + (k + i) * pitch)
                     : "memory");
    asm volatile("cp.async.wait_all;" ::: "memory");
    to = s_held + threadIdx.x;
    for (int k = 4 * kr; k < rows; k += kWk, to += 4 * kWeightThreads)
#pragma unroll
      for (int i = 0; i < 4; ++i) more(to[i * kWeightThreads]);
  } else {
#pragma unroll 8
    for (int k = kr; k < rows; k += kWeightThreads / 4) more(__ldcg(src + k * pitch));
  }
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) {  // the warp's eight rows
    m.x = __vmaxu2(m.x, __shfl_xor_sync(0xffffffffu, m.x, o));
    m.y = __vmaxu2(m.y, __shfl_xor_sync(0xffffffffu, m.y, o));
    m.z = __vmaxu2(m.z, __shfl_xor_sync(0xffffffffu, m.z, o));
    m.w = __vmaxu2(m.w, __shfl_xor_sync(0xffffffffu, m.w, o));
  }
  if (lane < 4) s_max[warp][lane] = m;
  __syncthreads();
  if constexpr (kWCtas == 1) {
    m = s_max[0][cg];
    for (int i = 1; i < kWeightThreads / 32; ++i) {
      const uint4 v = s_max[i][cg];
      m.x = __vmaxu2(m.x, v.x);
      m.y = __vmaxu2(m.y, v.y);
      m.z = __vmaxu2(m.z, v.z);
      m.w = __vmaxu2(m.w, v.w);
    }
  } else {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // every CTA has started
    if (threadIdx.x < 16) {  // a word of the 32 columns' maxima
      const uint32_t* word = reinterpret_cast<const uint32_t*>(s_max) + threadIdx.x;
      uint32_t mine = 0u;
      for (int i = 0; i < kWeightThreads / 32; ++i) mine = __vmaxu2(mine, word[16 * i]);
      const uint32_t* to = reinterpret_cast<const uint32_t*>(s_all[rank]) + threadIdx.x;
      for (uint32_t c = 0; c < kWCtas; ++c)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(map_to_cta(to, c)), "r"(mine) : "memory");
    }
    cluster_sync_all();
    m = s_all[0][cg];
#pragma unroll
    for (int i = 1; i < kWCtas; ++i) {
      const uint4 v = s_all[i][cg];
      m.x = __vmaxu2(m.x, v.x);
      m.y = __vmaxu2(m.y, v.y);
      m.z = __vmaxu2(m.z, v.z);
      m.w = __vmaxu2(m.w, v.w);
    }
  }
  float inv[8];
  uint32_t bad = 0u, raised = 0u;  // bit i: column 8 cg + i reads as NaN, is raised
  const uint32_t mw[4] = {m.x, m.y, m.z, m.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = (mw[i >> 1] >> (16 * (i & 1))) & 0xFFFFu;
    const float raise = raise_of(b);
    inv[i] = inverse_of(b, raise);
    if (b >= kInfBits) bad |= 1u << i;
    if (raise != 1.0f) raised |= 1u << i;
    if (kr == 0 && rank == 0) scales[e * N + n0 + 8 * cg + i] = scale_of(b);
  }
  const bool any_raised = __any_sync(0xffffffffu, raised != 0u);
  for (int k0 = (rows - 1) / kWk * kWk; k0 >= 0; k0 -= kWk) {
    const int k = k0 + 4 * kr;
    if (k < rows) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = kHeld ? s_held[(k0 / kWk * 4 + i) * kWeightThreads + threadIdx.x] : __ldcg(src + (k + i) * pitch);
      const uint32_t a[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // column 8 cg + i: its four k's are one word
        float f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = i & 1 ? bf16hi_to_f32(a[j][i >> 1]) : bf16lo_to_f32(a[j][i >> 1]);
        if (any_raised && ((raised >> i) & 1u)) {
          const float raise = inv[i] > 1.0f ? 0x1p64f : 0x1p-64f;
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] *= raise;
        }
        const uint32_t q =
            pack4(code_of(f[0] * inv[i]), code_of(f[1] * inv[i]), code_of(f[2] * inv[i]), code_of(f[3] * inv[i]));
        // 16-byte chunks of a column are permuted by its group, which spreads
        // both accesses over all banks
        const int chunk = (kr >> 2) ^ (2 * cg);
        s_codes[(8 * cg + i) * (kWk / 4) + chunk * 4 + (kr & 3)] = (bad >> i) & 1u ? 0u : q;
      }
    }
    __syncthreads();
    const int left = min(kWk, rows - k0) / 16;  // 16-byte chunks of a column
    for (int i = threadIdx.x; i < kWn * (kWk / 16); i += kWeightThreads) {
      const int n = i / (kWk / 16), c = i % (kWk / 16);
      if (c < left)
        *reinterpret_cast<uint4*>(codes + (e * N + n0 + n) * K + first + k0 + c * 16) =
            *reinterpret_cast<const uint4*>(s_codes + n * (kWk / 4) + (c ^ (2 * (n >> 3))) * 4);
    }
    __syncthreads();
  }
}

// The weights' kernel for a cluster of `ctas` CTAs.
using WeightsKernel = void (*)(const uint16_t*, int, int, int8_t*, float*);
WeightsKernel weights_kernel(int ctas, bool held) {
  return !held       ? quantize_weights_kernel<2, false>
         : ctas == 1 ? quantize_weights_kernel<1, true>
         : ctas == 2 ? quantize_weights_kernel<2, true>
         : ctas == 4 ? quantize_weights_kernel<4, true>
                     : quantize_weights_kernel<8, true>;
}

int group_of(int64_t cols) {
  int group = 1;
  while (group < 8 && cols > 32 * 8 * kRowVecs * group) group *= 2;
  return group;
}

}  // namespace

cudaError_t launch_quantize_rows_int8(const uint16_t* x, int64_t rows, int64_t cols, int8_t* codes, float* scales,
                                      cudaStream_t st) {
  const int group = group_of(cols);
  const int64_t per = 8 / group;
  return launch_pdl(quantize_rows_kernel, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(256), 0, st, x,
                    rows, static_cast<int>(cols), nullptr, 1, rows, nullptr, nullptr, group, codes, scales, nullptr);
}

cudaError_t launch_quantize_expert_rows_int8(const moe_shape& s, const uint16_t* x, int64_t cols,
                                             const int32_t* gather_idx, const int32_t* num_blocks, int8_t* codes,
                                             float* scales, cudaStream_t st) {
  const int group = group_of(cols);
  const int64_t per = 8 / group, rows = max_rows_of(s);
  return launch_pdl(quantize_rows_kernel, dim3(static_cast<unsigned>((rows + per - 1) / per)), dim3(256), 0, st, x,
                    rows, static_cast<int>(cols), nullptr, 1, rows, gather_idx, num_blocks, group, codes, scales,
                    nullptr);
}

cudaError_t launch_quantize_permute_int8(const moe_shape& s, const uint16_t* X, const int32_t* scatter_idx,
                                         int8_t* codes, float* scales, uint32_t* status, cudaStream_t st) {
  const int group = group_of(s.H);
  const int64_t per = 8 / group;
  return launch_pdl(quantize_rows_kernel, dim3(static_cast<unsigned>((s.T + per - 1) / per)), dim3(256), 0, st, X,
                    static_cast<int64_t>(s.T), s.H, scatter_idx, s.k, max_rows_of(s), nullptr, nullptr, group, codes,
                    scales, status);
}

cudaError_t launch_dequantize_rows_int8(const int8_t* codes, const float* scales, int64_t rows, int64_t cols,
                                        uint16_t* x, cudaStream_t st) {
  const int64_t n8 = rows * (cols / 8);
  constexpr int kPer = 256 * kDeqVecs;
  return launch_pdl(dequantize_rows_kernel, dim3(static_cast<unsigned>((n8 + kPer - 1) / kPer)), dim3(256), 0, st,
                    codes, scales, n8, static_cast<int>(cols / 8), x);
}

cudaError_t launch_quantize_weights_int8(const uint16_t* w, int E, int64_t K, int64_t N, int8_t* codes, float* scales,
                                         int num_sms, cudaStream_t st) {
  constexpr auto held_bytes = [](int64_t rows) { return (rows + kWk - 1) / kWk * 4 * kWeightThreads * 16; };
  // the shared-memory opt-in, once per device (host threads may race here)
  static bool done[64] = {};
  static std::mutex mu;
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (dev >= 64 || !done[dev]) {
      for (int ctas = 1; ctas <= 8 && err == cudaSuccess; ctas *= 2)
        err = cudaFuncSetAttribute(weights_kernel(ctas, true), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   static_cast<int>(held_bytes(kMostHeld)));
      if (err != cudaSuccess) return err;
      if (dev < 64) done[dev] = true;
    }
  }
  int ctas = 1;
  while (ctas < 8 && K > ctas * kMostHeld) ctas *= 2;
  const bool held = K <= ctas * kMostHeld;
  if (!held) ctas = 2;
  while (held && ctas < 4 && 2 * (N / kWn) * E * ctas <= 4 * num_sms) ctas *= 2;
  const WeightsKernel kernel = weights_kernel(ctas, held);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(N / kWn), static_cast<unsigned>(ctas), static_cast<unsigned>(E));
  cfg.blockDim = dim3(kWeightThreads);
  cfg.dynamicSmemBytes = held ? static_cast<size_t>(held_bytes(K / ctas)) : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 1;
  attr[0].val.clusterDim.y = static_cast<unsigned>(ctas);
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, w, static_cast<int>(K), static_cast<int>(N), codes, scales);
}

}  // namespace moe
