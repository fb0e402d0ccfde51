// moe_balance.cu -- the router's balance loss, its per-expert counts and the
// gradient to the logits.
//
// Over the n tokens that take part (mask byte non-zero, or no mask, and not
// every logit -inf), with p = softmax(logits), f_e = counts_e / (n k) and
// P_e = sum_t p_te / n:
//   balance = E sum_e f_e P_e          z = sum_t logsumexp(l_t)^2 / n
//   d/dl_te = p_te [ g0 E/n (f_e - sum_j f_j p_tj) + g1 2/n logsumexp(l_t) ]
// (the counts are constants for the gradient).  Both kernels read the logits
// once and are bound by memory on large batches and by launch latency on small
// ones: 262144 x 256 logits with 85% of the tokens taking part take 47 us
// forward (5.0 TB/s; 6.2 past a fixed 10 us of start and of joining the CTAs'
// sums) and 82 us backward (6.0 TB/s), 128 x 8 logits 3.0 and 2.1 us.  Until the
// lanes per token were fixed at compile time (unrolled exchanges) and exp, log
// and reciprocal left to the SFU they were bound by instructions (81 and 103 us).
//
// What a kernel of this library wrote just before (picks, counts, partial sums)
// is not read through the non-coherent path: under programmatic dependent launch
// a CTA may become resident before it is written.  Picks and counts are cached in
// L1 all the same (__ldca): every warp of the backward kernel reads all counts,
// and past L1 its smallest calls took a quarter longer, mid-sized ones three
// times as long.
//
// A token's row is held by a group of G lanes (a power of two up to 32), each
// with up to eight logits: groups of four consecutive ones (16-byte loads)
// where E is a multiple of 4, single ones otherwise.  Sums over tokens are
// kept per lane and joined in a fixed order (warp, CTA, then the CTA that
// finishes last over all CTAs), so results are reproducible without
// floating-point atomics.
#include <cmath>
#include <cstdint>

#include "moe_device.cuh"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kMaxE = 256;
constexpr int kFwdThreads = 1024;
constexpr int kFwdWarps = kFwdThreads / 32;
constexpr int kBwdThreads = 256;

// e^x and ln(x) on the SFU; e^x below the smallest normal float is 0.
__device__ __forceinline__ float fast_exp(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x * 1.4426950408889634f));
  return r;
}
__device__ __forceinline__ float fast_log(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r * 0.6931471805599453f;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Maximum and sum over the G lanes of a group (all 32 lanes call them).
template <int G>
__device__ __forceinline__ float group_max(float x) {
  if constexpr (G == 32) {
    float r;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
  } else {
#pragma unroll
    for (int o = G / 2; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
  }
}
template <int G>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// A lane's logits of one row: V groups of W consecutive experts, group i of
// lane gl (its index inside its G lanes) at expert W (gl + G i).
template <int V, int W, int G>
struct Row {
  float v[V * W];

  __device__ __forceinline__ static int expert(int gl, int x) { return W * (gl + G * (x / W)) + x % W; }

  // `row`: the lane's first logit; absent experts (and whole rows that are
  // not `there`) read as -inf
  __device__ __forceinline__ void load(const float* __restrict__ row, int gl, int E, bool there) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool in = there && W * (gl + G * i) < E;
      if constexpr (W == 4) {
        float4 q = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (in) q = __ldcg(reinterpret_cast<const float4*>(row + 4 * G * i));
        v[4 * i] = q.x;
        v[4 * i + 1] = q.y;
        v[4 * i + 2] = q.z;
        v[4 * i + 3] = q.w;
      } else {
        v[i] = in ? __ldcg(row + G * i) : -INFINITY;
      }
    }
  }

  // v becomes exp(v - max) (max taken as 0 where nothing is above -inf);
  // returns that max and the row's sum, which is 0 only if every logit is
  // -inf (a NaN anywhere makes it NaN).
  __device__ __forceinline__ void exps(float& top, float& sum) {
    float m = v[0];
#pragma unroll
    for (int x = 1; x < V * W; ++x) m = fmaxf(m, v[x]);
    m = group_max<G>(m);
    top = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int x = 0; x < V * W; ++x) {
      v[x] = fast_exp(v[x] - top);
      s += v[x];
    }
    sum = group_sum<G>(s);
  }
};

// Rows each group of lanes has in flight at a time.  (262144 x 256 forward: one
// 54 us, two 47 us, three or four with fewer threads for the registers 52 and
// 63 us; rows copied ahead to shared memory 61 us.)
constexpr int kUnroll = 2;

template <int V, int W, int G>
__global__ void __launch_bounds__(kFwdThreads, 1)
    balance_loss_kernel(const float* __restrict__ logits, const int32_t* __restrict__ topk_ids,
                        const uint8_t* __restrict__ mask, int T, int E, int k, int32_t* __restrict__ counts,
                        int32_t* __restrict__ num_tokens, float* __restrict__ mean_probs, float* __restrict__ losses,
                        uint32_t* __restrict__ partials, uint32_t* __restrict__ counter,
                        uint32_t* __restrict__ status) {
  __shared__ __align__(16) float s_p[kFwdWarps * kMaxE];
  __shared__ int s_cnt[kMaxE];
  __shared__ float s_z[kFwdWarps];
  __shared__ int s_n[kFwdWarps];
  __shared__ int s_last;
  pdl_launch_dependents();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gl = lane & (G - 1);
  constexpr int per_warp = 32 / G;
  for (int e = tid; e < E; e += kFwdThreads) s_cnt[e] = 0;
  __syncthreads();
  pdl_wait();

  float acc[V * W];
#pragma unroll
  for (int x = 0; x < V * W; ++x) acc[x] = 0.0f;
  float z = 0.0f;
  int n = 0;
  const int64_t step = static_cast<int64_t>(per_warp) * kUnroll;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kFwdWarps * step;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kFwdWarps + warp) * step + lane / G;
  const int64_t warp_first = first - lane / G;
  // Where a token has as many lanes as picks can be, lane gl counts pick gl.
  // Otherwise the picks of a row step's per_warp tokens, per_warp k consecutive
  // ints, go round the warp's lanes (k <= E <= W G, so at most W each): tok is
  // the token of the step that each is of.
  constexpr bool kSpread = G < 16;
  constexpr int kPicks = kSpread ? W : 1;
  int tok[kPicks];
#pragma unroll
  for (int q = 0; q < kPicks; ++q) {
    tok[q] = per_warp;  // none
    if (kSpread ? 32 * q < per_warp * k : gl < k) tok[q] = kSpread ? (lane + 32 * q) / k : lane / G;
  }
  // the masks are read one iteration ahead of the rows they decide on
  bool use[kUnroll];
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const int64_t t = first + u * per_warp;
    use[u] = t < T && (mask == nullptr || __ldca(mask + t) != 0);
  }
  for (int64_t d = 0; warp_first + d < T; d += stride) {  // uniform across the warp
    Row<V, W, G> r[kUnroll];
    int id[kUnroll][kPicks];
    bool there[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t t = first + d + u * per_warp;
      there[u] = use[u];
      r[u].load(logits + t * E + W * gl, gl, E, there[u]);
      const int64_t t0 = warp_first + d + u * per_warp;
#pragma unroll
      for (int q = 0; q < kPicks; ++q) {
        id[u][q] = 0;
        if (kSpread && 32 * q >= per_warp * k) break;  // uniform
        if constexpr (kSpread)
          id[u][q] = tok[q] < per_warp && t0 + tok[q] < T ? __ldca(topk_ids + t0 * k + lane + 32 * q) : 0;
        else
          id[u][q] = there[u] && gl < k ? __ldca(topk_ids + t * k + gl) : 0;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t t = first + d + stride + u * per_warp;
      use[u] = t < T && (mask == nullptr || __ldca(mask + t) != 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      float top, sum;
      r[u].exps(top, sum);
      const bool takes = there[u] && sum != 0.0f;
      const uint32_t who = kSpread ? __ballot_sync(0xffffffffu, takes) : 0u;
#pragma unroll
      for (int q = 0; q < kPicks; ++q) {
        if (kSpread && 32 * q >= per_warp * k) break;
        if (tok[q] >= per_warp || !(kSpread ? (who >> (tok[q] * G)) & 1u : takes)) continue;
        const int e = id[u][q];
        if (static_cast<unsigned>(e) < static_cast<unsigned>(E)) atomicAdd(&s_cnt[e], 1);
        else record_status(status, kStatusBounds);
      }
      if (!takes) continue;
      const float inv = fast_rcp(sum);
#pragma unroll
      for (int x = 0; x < V * W; ++x) acc[x] += r[u].v[x] * inv;
      if (gl == 0) {
        const float lse = top + fast_log(sum);
        z += lse * lse;
        ++n;
      }
    }
  }
  // the warp's groups hold the same experts: join them, then the warps
  for (int o = G; o < 32; o <<= 1) {
#pragma unroll
    for (int x = 0; x < V * W; ++x) acc[x] += __shfl_xor_sync(0xffffffffu, acc[x], o);
  }
  for (int o = 16; o > 0; o >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, o);
    n += __shfl_xor_sync(0xffffffffu, n, o);
  }
  if (lane < G) {
#pragma unroll
    for (int x = 0; x < V * W; ++x) {
      const int e = Row<V, W, G>::expert(gl, x);
      if (e < E) s_p[warp * E + e] = acc[x];
    }
  }
  if (lane == 0) {
    s_z[warp] = z;
    s_n[warp] = n;
  }
  __syncthreads();
  float p_sum = 0.0f;  // thread e < E: this CTA's sum for expert e
  int c_sum = 0;
  if (tid < E) {
    for (int w = 0; w < kFwdWarps; ++w) p_sum += s_p[w * E + tid];
    c_sum = s_cnt[tid];
  }
  float z_sum = 0.0f;  // warp 0: the CTA's
  int n_sum = 0;
  if (warp == 0) {
    z_sum = s_z[lane];
    n_sum = s_n[lane];
    for (int o = 16; o > 0; o >>= 1) {
      z_sum += __shfl_xor_sync(0xffffffffu, z_sum, o);
      n_sum += __shfl_xor_sync(0xffffffffu, n_sum, o);
    }
  }

  if (gridDim.x > 1) {
    // partials: [CTA][E] sums, [CTA][E] counts, [CTA] z, [CTA] n
    float* part_p = reinterpret_cast<float*>(partials);
    int32_t* part_c = reinterpret_cast<int32_t*>(partials) + static_cast<int64_t>(gridDim.x) * E;
    float* part_z = reinterpret_cast<float*>(part_c + static_cast<int64_t>(gridDim.x) * E);
    int32_t* part_n = reinterpret_cast<int32_t*>(part_z + gridDim.x);
    if (tid < E) {
      part_p[blockIdx.x * E + tid] = p_sum;
      part_c[blockIdx.x * E + tid] = c_sum;
    }
    if (tid == 0) {
      part_z[blockIdx.x] = z_sum;
      part_n[blockIdx.x] = n_sum;
    }
    __syncthreads();
    if (tid == 0) {
      fence_acq_rel_gpu();  // release: the CTA's partials (ordered by the barrier) before the arrival
      // The word counts the CTAs that have arrived (bits 0-9) and sums their
      // indexes plus one above.  The last one is known by the sum; c of them
      // cannot sum to less than c (c + 1) / 2, and only the whole grid sums to
      // `all`: anything else was in the word before the launch (a leftover that
      // is itself the state of some CTAs' arrivals is not told from them).
      const uint32_t mine = 1u | ((blockIdx.x + 1u) << 10);
      const uint32_t seen = atomicAdd(counter, mine) + mine;
      const uint32_t c = seen & 0x3FFu, sum = seen >> 10, all = gridDim.x * (gridDim.x + 1u) / 2u;
      if (sum < c * (c + 1u) / 2u || sum > all || (sum == all) != (c == gridDim.x))
        record_status(status, kStatusBounds);
      s_last = sum == all ? 1 : 0;
      if (sum >= all) *counter = 0u;
      fence_acq_rel_gpu();  // acquire: every other CTA's partials
    }
    __syncthreads();
    if (!s_last) return;
    // the CTAs' rows of partials go round `parts` groups of threads, a thread
    // to W neighbouring experts; the groups' sums join in a fixed order
    const int cols = (E + W - 1) / W;  // E % 4 == 0 where W is 4
    const int parts = min(32, min(kFwdThreads / cols, kFwdWarps * kMaxE / 2 / E));
    const int part = tid / cols, e = tid % cols * W;
    int* s_ci = reinterpret_cast<int*>(s_p) + kFwdWarps * kMaxE / 2;
    constexpr int kRows = V * W > 4 ? 3 : 5;  // in flight per thread, as registers allow
    if (part < parts) {
      float ps[W];
      int cs[W];
#pragma unroll
      for (int q = 0; q < W; ++q) {
        ps[q] = 0.0f;
        cs[q] = 0;
      }
#pragma unroll kRows
      for (int b = part; b < static_cast<int>(gridDim.x); b += parts) {
        if constexpr (W == 4) {
          const float4 p4 = __ldcg(reinterpret_cast<const float4*>(part_p + b * E + e));
          const int4 c4 = __ldcg(reinterpret_cast<const int4*>(part_c + b * E + e));
          ps[0] += p4.x; ps[1] += p4.y; ps[2] += p4.z; ps[3] += p4.w;
          cs[0] += c4.x; cs[1] += c4.y; cs[2] += c4.z; cs[3] += c4.w;
        } else {
          ps[0] += __ldcg(part_p + b * E + e);
          cs[0] += __ldcg(part_c + b * E + e);
        }
      }
#pragma unroll
      for (int q = 0; q < W; ++q) {
        s_p[part * E + e + q] = ps[q];
        s_ci[part * E + e + q] = cs[q];
      }
    }
    if (warp == 0) {
      z_sum = 0.0f;
      n_sum = 0;
      for (int b = lane; b < static_cast<int>(gridDim.x); b += 32) {
        z_sum += __ldcg(part_z + b);
        n_sum += __ldcg(part_n + b);
      }
      for (int o = 16; o > 0; o >>= 1) {
        z_sum += __shfl_xor_sync(0xffffffffu, z_sum, o);
        n_sum += __shfl_xor_sync(0xffffffffu, n_sum, o);
      }
    }
    __syncthreads();
    if (tid < E) {
      p_sum = 0.0f;
      c_sum = 0;
      for (int q = 0; q < parts; ++q) {
        p_sum += s_p[q * E + tid];
        c_sum += s_ci[q * E + tid];
      }
    }
    __syncthreads();
  }
  // the results: thread e writes its expert's; warps 0-7 form the dot product
  if (tid == 0) s_n[0] = n_sum;
  __syncthreads();
  const int total_n = s_n[0];
  const float inv_n = total_n > 0 ? 1.0f / static_cast<float>(total_n) : 0.0f;
  float dot = 0.0f;
  if (tid < E) {
    const float P = p_sum * inv_n;
    counts[tid] = c_sum;
    mean_probs[tid] = P;
    dot = total_n > 0 ? static_cast<float>(c_sum) / (static_cast<float>(total_n) * static_cast<float>(k)) * P : 0.0f;
  }
  if (warp < kMaxE / 32) {
    for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
    if (lane == 0) s_z[warp] = dot;
  }
  __syncthreads();
  if (tid == 0) {
    float d = 0.0f;
    for (int w = 0; w < kMaxE / 32; ++w) d += s_z[w];
    losses[0] = static_cast<float>(E) * d;
    losses[1] = z_sum * inv_n;
    *num_tokens = total_n;
  }
}

template <int V, int W, int G>
__global__ void __launch_bounds__(kBwdThreads)
    balance_backward_kernel(const float* __restrict__ logits, const uint8_t* __restrict__ mask, int T, int E, int k,
                            const int32_t* __restrict__ counts, const int32_t* __restrict__ num_tokens,
                            const float* __restrict__ grad_losses, float* __restrict__ dlogits) {
  pdl_launch_dependents();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int gl = lane & (G - 1);
  constexpr int per_warp = 32 / G;
  constexpr int kWarps = kBwdThreads / 32;
  const int n = __ldca(num_tokens);
  const float inv_n = n > 0 ? 1.0f / static_cast<float>(n) : 0.0f;
  const float a = __ldca(grad_losses) * static_cast<float>(E) * inv_n;
  const float b = __ldca(grad_losses + 1) * 2.0f * inv_n;
  // f_e - 1/E, whose differences are the gradient's: formed from integers, so
  // that f_e - sum f p loses nothing to cancellation (the p sum to 1)
  float f[V * W];
#pragma unroll
  for (int x = 0; x < V * W; ++x) {
    const int e = Row<V, W, G>::expert(gl, x);
    f[x] = 0.0f;
    if (e < E && n > 0) {
      const int64_t nk = static_cast<int64_t>(n) * k;
      f[x] = static_cast<float>(static_cast<int64_t>(__ldca(counts + e)) * E - nk) /
             (static_cast<float>(nk) * static_cast<float>(E));
    }
  }
  // from the last token to the first: the logits that the forward pass read
  // last are the ones that L2 still holds
  const int64_t step = static_cast<int64_t>(per_warp) * kUnroll;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps * step;
  const int64_t tiles = (T + step - 1) / step;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < tiles; i += stride / step) {
    const int64_t t0 = (tiles - 1 - i) * step + lane / G;
    Row<V, W, G> r[kUnroll];
    bool there[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t t = t0 + u * per_warp;
      there[u] = t < T && (mask == nullptr || __ldca(mask + t) != 0);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) r[u].load(logits + (t0 + u * per_warp) * E + W * gl, gl, E, there[u]);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int64_t t = t0 + u * per_warp;
      float top, sum;
      r[u].exps(top, sum);
      const bool takes = there[u] && sum != 0.0f;
      const float inv = fast_rcp(sum);
      float dot = 0.0f;
#pragma unroll
      for (int x = 0; x < V * W; ++x) dot = fmaf(f[x], r[u].v[x], dot);
      dot = group_sum<G>(dot) * inv;
      if (t >= T) continue;
      // p (a f + c) with p = v / sum
      const float ia = a * inv;
      const float ic = (b * (top + fast_log(sum)) - a * dot) * inv;
      float* out = dlogits + t * E + W * gl;
#pragma unroll
      for (int x = 0; x < V; ++x) {
        if (W * (gl + G * x) >= E) continue;
        float d[W];
#pragma unroll
        for (int q = 0; q < W; ++q) d[q] = takes ? r[u].v[W * x + q] * fmaf(ia, f[W * x + q], ic) : 0.0f;
        if constexpr (W == 4) *reinterpret_cast<float4*>(out + 4 * G * x) = make_float4(d[0], d[1], d[2], d[3]);
        else out[G * x] = d[0];
      }
    }
  }
}

// Calls fn with the row split of E experts: as few logits per lane and lanes
// per token as cover E.
template <int V, int W, int G>
struct Split {};
template <int W, int G = 1, typename F>
cudaError_t by_lanes(int E, F&& fn) {
  if constexpr (G < 32) {
    if (E > W * G) return by_lanes<W, 2 * G>(E, fn);
  }
  return fn(Split<1, W, G>{});
}
template <typename F>
cudaError_t by_experts(int E, F&& fn) {
  if (E % 4 == 0) return E <= 128 ? by_lanes<4>(E, fn) : fn(Split<2, 4, 32>{});
  if (E <= 32) return by_lanes<1>(E, fn);
  if (E <= 64) return fn(Split<2, 1, 32>{});
  return E <= 128 ? fn(Split<4, 1, 32>{}) : fn(Split<8, 1, 32>{});
}

template <int V, int W, int G>
cudaError_t loss_call(Split<V, W, G>, const moe_shape& s, const float* logits, const int32_t* topk_ids,
                      const uint8_t* mask, int32_t* counts, int32_t* num_tokens, float* mean_probs, float* losses,
                      uint32_t* partials, uint32_t* counter, uint32_t* status, int num_sms, cudaStream_t st) {
  constexpr int kPerCta = kFwdWarps * (32 / G) * kUnroll;
  int grid = (s.T + kPerCta - 1) / kPerCta;
  if (grid > num_sms) grid = num_sms;
  if (grid > kBalanceMaxCtas) grid = kBalanceMaxCtas;
  return launch_pdl(balance_loss_kernel<V, W, G>, dim3(grid), dim3(kFwdThreads), 0, st, logits, topk_ids, mask, s.T,
                    s.E, s.k, counts, num_tokens, mean_probs, losses, partials, counter, status);
}

template <int V, int W, int G>
cudaError_t backward_call(Split<V, W, G>, const moe_shape& s, const float* logits, const uint8_t* mask,
                          const int32_t* counts, const int32_t* num_tokens, const float* grad_losses, float* dlogits,
                          int num_sms, cudaStream_t st) {
  constexpr int kPerCta = kBwdThreads / 32 * (32 / G) * kUnroll;
  int grid = (s.T + kPerCta - 1) / kPerCta;
  if (grid > num_sms * 8) grid = num_sms * 8;
  return launch_pdl(balance_backward_kernel<V, W, G>, dim3(grid), dim3(kBwdThreads), 0, st, logits, mask, s.T, s.E,
                    s.k, counts, num_tokens, grad_losses, dlogits);
}

}  // namespace

cudaError_t launch_balance_loss(const moe_shape& s, const float* logits, const int32_t* topk_ids, const uint8_t* mask,
                                int32_t* counts, int32_t* num_tokens, float* mean_probs, float* losses,
                                uint32_t* partials, uint32_t* counter, uint32_t* status, int num_sms,
                                cudaStream_t st) {
  return by_experts(s.E, [&](auto split) {
    return loss_call(split, s, logits, topk_ids, mask, counts, num_tokens, mean_probs, losses, partials, counter,
                     status, num_sms, st);
  });
}

cudaError_t launch_balance_backward(const moe_shape& s, const float* logits, const uint8_t* mask,
                                    const int32_t* counts, const int32_t* num_tokens, const float* grad_losses,
                                    float* dlogits, int num_sms, cudaStream_t st) {
  return by_experts(s.E, [&](auto split) {
    return backward_call(split, s, logits, mask, counts, num_tokens, grad_losses, dlogits, num_sms, st);
  });
}

}  // namespace moe
