/*
 * moe.h -- C ABI of the GB300 (sm_103a) Mixture-of-Experts expert layer.
 *
 * The layer, per token t with router logits l[t, :] over E experts:
 *   1. route:   softmax over the E logits, the k largest picked (ties to the
 *               lower expert index, slot j = j-th pick), weights renormalised
 *               over the picks;
 *   2. permute: the T*k routed rows grouped by expert into 128-row blocks
 *               (each expert's group padded to a multiple of 128 rows),
 *               tokens ascending inside an expert;
 *   3. up:      per block of expert e, h = bf16(SiLU(A Wg[e]) * (A Wu[e]));
 *   4. down:    Y = bf16(h Wd[e]);
 *   5. combine: out[t] = bf16(sum_j w[t,j] * Y[row(t,j)]), float32, slot order.
 * Sources: "通算融合算子（一）：为什么要把通信写进 GEMM kernel 里" §1 (the serial
 * layer: gate/up GEMM -> SiLU -> down GEMM) and §4 (table of data-flow
 * patterns: "dispatch + GEMM" reorders rows by the route, "GEMM + combine" is
 * the top-k weighted reduction); "通算融合算子（三）：ThunderKittens 多卡编程与
 * 可融合的 GEMM 模板" §4 (grouped GEMM over expert row blocks of 128 rows, 128 =
 * expert alignment unit, expert-major task order).
 *
 * Conventions for every call below:
 *   - all tensor pointers are DEVICE pointers, 16-byte aligned, dense
 *     row-major; bf16 tensors are passed as raw 16-bit patterns (moe_bf16);
 *   - the caller owns every buffer; the library allocates no device memory;
 *   - calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and never synchronise, except moe_workspace_size,
 *     moe_capacity (host only) and moe_last_device_status (synchronises);
 *   - argument and shape errors are returned before anything is launched;
 *     a failed launch returns MOE_ERR_CUDA; errors found by the kernels
 *     themselves (a bounded wait that ran out, an index out of range) are
 *     recorded in the workspace status word and reported by
 *     moe_last_device_status;
 *   - results are bitwise reproducible run to run (no floating-point atomics);
 *   - the step calls and moe_forward may be recorded into a CUDA graph by
 *     stream capture (they only launch kernels on `stream`; the launches keep
 *     their programmatic-dependent-launch edges); moe_last_device_status
 *     synchronises and is not capturable;
 *   - the device must have compute capability 10.3 (GB300), else MOE_ERR_ARCH;
 *   - a call makes the stream's device current for its launches and puts the
 *     calling thread's previous current device back before it returns.
 *
 * The experts' products also run on MXFP4 operands (moe_*_mxfp4) and on 8-bit
 * integers (moe_*_int8), the router's balance loss has its gradient
 * (moe_balance_loss*), and the layer has its backward pass (moe_forward_train,
 * moe_*backward); each is described where it is declared.
 *
 * Supported shapes (else MOE_ERR_UNSUPPORTED_SHAPE): 1 <= T <= 2^22,
 * 1 <= E <= 256, 1 <= k <= min(E, 16), 128 <= H <= 32768 and
 * 128 <= I <= 32768 with H % 128 == 0 and I % 128 == 0.
 *
 * Capacity: max_blocks = (T*k + 127*min(E, T*k)) / 128 bounds the number of
 * 128-row blocks of any routing; max_rows = 128 * max_blocks.  Buffers indexed
 * by permuted row (gather_idx, h, Y) hold max_rows rows; block_expert holds
 * max_blocks entries.  Only the first num_blocks (device value) blocks are
 * meaningful; entries past them are left unwritten.
 */
#ifndef MOE_GB300_H
#define MOE_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t moe_bf16;                 /* raw bfloat16 bits */
typedef struct CUstream_st *moe_stream_t;  /* == cudaStream_t */

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = 1,        /* NULL pointer or NULL shape */
    MOE_ERR_UNSUPPORTED_SHAPE = 2,  /* shape outside the supported range */
    MOE_ERR_MISALIGNED = 3,         /* a pointer is not 16-byte aligned */
    MOE_ERR_ARCH = 4,               /* device is not compute capability 10.3 */
    MOE_ERR_CUDA = 5,               /* a CUDA runtime call or launch failed */
    MOE_ERR_TIMEOUT = 6,            /* a kernel's bounded wait ran out */
    MOE_ERR_DEVICE_BOUNDS = 7,      /* a kernel met an index out of range */
    MOE_ERR_SCRATCH_LIMIT = 8       /* moe_route_noalloc: shape needs more than its fixed scratch */
} moe_status;

typedef struct {
    int32_t T;  /* tokens */
    int32_t H;  /* hidden size */
    int32_t I;  /* expert intermediate size */
    int32_t E;  /* experts */
    int32_t k;  /* experts per token */
} moe_shape;

/* Human-readable name of a status code (static storage). */
const char *moe_status_string(moe_status s);

/* Host only.  Writes max_blocks and max_rows (see Capacity above). */
moe_status moe_capacity(const moe_shape *shape, int64_t *max_blocks, int64_t *max_rows);

/* Host only.  Bytes of the workspace `ws` that every call below accepts
 * (the largest need, that of moe_forward).  One workspace serves all calls
 * of one shape; calls sharing it must be ordered on one stream. */
moe_status moe_workspace_size(const moe_shape *shape, size_t *bytes);

/* Clears the first 256 bytes of `ws`: the status word, the routing's chunk
 * counter and scan mark, both GEMMs' tile counters and the slot where each
 * forward records the status it started with.  Call once after allocating `ws` (asynchronous,
 * on `stream`); the kernels leave their counters cleared for the next call.
 * On a workspace that was never cleared the routing may scan its histograms
 * early and a GEMM may skip tiles; each reports MOE_ERR_DEVICE_BOUNDS when a
 * counter is out of range, and the next call finds the counters cleared.  (The per-window counts of moe_forward, further
 * on in `ws`, are cleared by every forward itself.) */
moe_status moe_workspace_init(const moe_shape *shape, void *ws, moe_stream_t stream);

/* Synchronises `stream`, returns the error recorded by the kernels since the
 * last call (MOE_OK if none) and clears it. */
moe_status moe_last_device_status(void *ws, moe_stream_t stream);

/* Diagnostic for the kernels' bounded waits: launches one thread that waits
 * on an mbarrier nothing arrives on, through the same bounded wait as every
 * pipeline of the library.  After the wait limit (2 s) the kernel records a
 * timeout in the status word at the start of `ws` (a workspace, or any 16-byte
 * aligned device buffer of at least 4 bytes whose first word is the status
 * word) and returns; the GPU is not faulted.  The next
 * moe_last_device_status(ws) returns MOE_ERR_TIMEOUT.  Asynchronous like the
 * step calls; the stream is busy for about 2 s. */
moe_status moe_check_wait_timeout(void *ws, moe_stream_t stream);

/* Steps 1-2: routing, histogram, padded block table and permutation.
 * Passages: "通算融合算子（一）：为什么要把通信写进 GEMM kernel 里" §4, table row
 * "dispatch + GEMM" (the routed rows are reordered by the route before the
 * GEMM); "Lecture 11: Programming Systems for Specialized Hardware" example 4
 * (softmax as exp -> sum -> divide); "通算融合算子（三）：ThunderKittens 多卡编程与
 * 可融合的 GEMM 模板" §4 (128 rows = task block = expert alignment unit).
 *   logits       [T, E]  float32 (finite values)
 *   topk_ids     [T, k]  int32  out: picked experts, slot order
 *   topk_w       [T, k]  float32 out: renormalised weights
 *   counts       [E]     int32  out: rows per expert
 *   off_pad      [E+1]   int32  out: first padded row of each expert, off_pad[E] = 128*num_blocks
 *   block_expert [max_blocks] int32 out: expert of each 128-row block
 *   num_blocks   [1]     int32  out: number of blocks (stays on the device)
 *   gather_idx   [max_rows] int32 out: token of each permuted row, -1 for padding
 *   scatter_idx  [T, k]  int32  out: permuted row of each (token, slot)
 *   ws           workspace (scratch: per-chunk expert histograms; the chunk
 *                counter in its cleared first 256 bytes)
 * Counts, table and permutation are exact; topk_ids are exact for the
 * float32 logits given; topk_w is within a few float32 ulps of the
 * correctly rounded value. */
moe_status moe_route(const moe_shape *shape, const float *logits,
                     int32_t *topk_ids, float *topk_w, int32_t *counts,
                     int32_t *off_pad, int32_t *block_expert, int32_t *num_blocks,
                     int32_t *gather_idx, int32_t *scatter_idx, void *ws,
                     moe_stream_t stream);

/* moe_route without a workspace: the same kernels and the same outputs as
 * moe_route, but the per-chunk expert histograms live in a fixed scratch
 * array that the library places in device memory when it is loaded, so the
 * caller passes only the inputs and outputs and nothing is allocated.  For
 * callers that are not allowed to allocate device memory: a plugin whose host
 * framework owns all device memory and hands it only its inputs and outputs,
 * or a deployment that reserves its memory up front and forbids allocation
 * once running (cudaMalloc may also synchronise the device and stall other
 * streams).  The pages describe no such variant; it has no counterpart there.
 *   - Limit: E * ceil(T/32) <= 262144 (1 MiB of int32 histograms, plus 256
 *     bytes for two counter words; e.g. E=128 with T up to 65536, E=256 with T up to
 *     32768); larger shapes return MOE_ERR_SCRATCH_LIMIT and launch nothing.
 *   - The scratch is one array per device, shared by every call and held
 *     until the process exits.  Calls whose work may overlap on the GPU (on
 *     different streams without ordering) race on it; order them on one
 *     stream.  Every histogram entry a call reads is written earlier in the
 *     same call, and the counter that must start at zero is zero when the
 *     library is loaded and is put back to zero by every call (the scan
 *     mark beside it is cleared at the start of every call), so nothing
 *     needs clearing between calls.
 *   - The first call on a device looks up the scratch address on that device
 *     (a host-side query, no allocation) and caches it.  That lookup may load
 *     the library's module on the device, so make the first call on each
 *     device before capturing any stream into a CUDA graph.
 *   - Kernel-side errors are not reported (there is no status word).
 * Arguments as moe_route, without ws. */
moe_status moe_route_noalloc(const moe_shape *shape, const float *logits,
                             int32_t *topk_ids, float *topk_w, int32_t *counts,
                             int32_t *off_pad, int32_t *block_expert, int32_t *num_blocks,
                             int32_t *gather_idx, int32_t *scatter_idx,
                             moe_stream_t stream);

/* Step 3: grouped gate/up GEMM with the SiLU(gate)*up epilogue.
 * Passages: "通算融合算子（三）：ThunderKittens 多卡编程与可融合的 GEMM 模板" §4
 * (grouped GEMM: each expert's rows multiply that expert's weights, tasks in
 * expert order); "通算融合算子（一）：为什么要把通信写进 GEMM kernel 里" §1 (gate/up
 * GEMM followed by SiLU; fused here into the GEMM's epilogue).
 * The GEMM finds each expert's rows from counts and off_pad (rows off_pad[e]
 * .. off_pad[e] + counts[e]) instead of from the block table, and cuts them
 * into windows of at most 256 rows; block_expert and num_blocks are not read.
 *   X          [T, H] bf16 tokens
 *   scatter_idx, counts, off_pad: moe_route's outputs; the call first copies
 *              X[t] to permuted row scatter_idx[t, j] of a workspace buffer
 *              (token by token, so each row of X is read once), then runs
 *              the GEMM over each expert's rows
 *   W_gate [E, H, I] bf16,  W_up [E, H, I] bf16
 *   h          [max_rows, I] bf16 out: h[r] = bf16(silu(g) * u) for every real
 *              row r (gather_idx[r] >= 0); padding rows hold values of no
 *              meaning (never read by the combine)
 *   ws         workspace (scratch: the gathered activation rows; the tile
 *              counter the kernel's clusters draw their tiles from)
 * g and u accumulate in float32 on the tensor cores; SiLU*up is formed in
 * float32 and rounded once to bf16. */
moe_status moe_grouped_gemm_up(const moe_shape *shape, const moe_bf16 *X,
                               const int32_t *scatter_idx, const int32_t *counts,
                               const int32_t *off_pad, const moe_bf16 *W_gate,
                               const moe_bf16 *W_up, moe_bf16 *h, void *ws,
                               moe_stream_t stream);

/* Step 3 on rows already grouped by expert (for callers whose dispatch
 * delivers them that way, as the expert-parallel dispatch of "通算融合算子（一）"
 * §4 does): the same GEMM and epilogue as moe_grouped_gemm_up, without the
 * row gather.
 *   Xp         [max_rows, H] bf16: row r holds the token of permuted row r
 *              (the rows of expert e from off_pad[e], counts[e] of them;
 *              padding rows are not read into any stored result)
 *   counts, off_pad, W_gate, W_up, h: as for moe_grouped_gemm_up
 *   ws         workspace (the tile counter, the status word) */
moe_status moe_grouped_gemm_up_rows(const moe_shape *shape, const moe_bf16 *Xp,
                                    const int32_t *counts, const int32_t *off_pad,
                                    const moe_bf16 *W_gate, const moe_bf16 *W_up,
                                    moe_bf16 *h, void *ws, moe_stream_t stream);

/* Step 4: grouped down GEMM.
 * Passages: "通算融合算子（三）：ThunderKittens 多卡编程与可融合的 GEMM 模板" §4 (the
 * same grouped GEMM); "通算融合算子（一）：为什么要把通信写进 GEMM kernel 里" §1 (the
 * down GEMM after SiLU).  Like the gate/up call it takes counts and off_pad in
 * place of the block table.
 *   h      [max_rows, I] bf16 (permuted rows), counts / off_pad from moe_route,
 *   W_down [E, I, H] bf16
 *   Y      [max_rows, H] bf16 out: Y[r] = bf16(h[r] W_down[expert of r]) for
 *          every real row r; padding rows hold values of no meaning */
moe_status moe_grouped_gemm_down(const moe_shape *shape, const moe_bf16 *h,
                                 const int32_t *counts, const int32_t *off_pad,
                                 const moe_bf16 *W_down, moe_bf16 *Y, void *ws,
                                 moe_stream_t stream);

/* Step 5: top-k weighted combine back to token order, without atomics.
 * Passage: "通算融合算子（一）：为什么要把通信写进 GEMM kernel 里" §4, table row
 * "GEMM + combine" (the epilogue's top-k weighted reduction).
 *   out[t, c] = bf16(sum_{j<k} topk_w[t,j] * Y[scatter_idx[t,j], c])
 * with a float32 accumulator in slot order, each product and each sum rounded
 * to float32 (no fused multiply-add).
 *   Y [max_rows, H] bf16, scatter_idx [T, k] int32, topk_w [T, k] float32,
 *   out [T, H] bf16; ws: workspace for the status word, or NULL (a row
 *   index outside [0, max_rows) then contributes zero without a report) */
moe_status moe_combine(const moe_shape *shape, const moe_bf16 *Y,
                       const int32_t *scatter_idx, const float *topk_w,
                       moe_bf16 *out, void *ws, moe_stream_t stream);

/* Steps 1-5 on one stream with no host synchronisation in between; all
 * intermediates live in `ws` (see moe_workspace_views).  Passages: those of
 * the five steps above; the per-window hand-off below follows the gate /
 * epilogue hooks of "通算融合算子（三）" §4 (a producer signals a counter per row
 * block, a consumer waits on it) inside one GPU.  Unlike the step
 * calls, which start each kernel after the previous one has completed, the
 * down GEMM here starts on each expert's token window as soon as every
 * gate/up tile of that window is stored (a per-window count kept in `ws`,
 * cleared by the row gather of each forward), so it fills the SMs the gate/up
 * GEMM frees.  The output is bit-identical to the step calls'. */
moe_status moe_forward(const moe_shape *shape, const float *logits, const moe_bf16 *X,
                       const moe_bf16 *W_gate, const moe_bf16 *W_up,
                       const moe_bf16 *W_down, moe_bf16 *out, void *ws,
                       moe_stream_t stream);

/* Device pointers to the intermediates that moe_forward leaves in `ws`
 * (valid after the forward's work on the stream has completed).  `ws` has
 * moe_workspace_size bytes: the smaller workspace of moe_forward_mxfp4 is laid
 * out otherwise, and the call cannot tell. */
typedef struct {
    int32_t *topk_ids;
    float *topk_w;
    int32_t *counts;
    int32_t *off_pad;
    int32_t *block_expert;
    int32_t *num_blocks;
    int32_t *gather_idx;
    int32_t *scatter_idx;
    moe_bf16 *h;
    moe_bf16 *Y;
    moe_bf16 *Xp;   /* [max_rows, H]: the gathered token rows in expert order */
} moe_views;

moe_status moe_workspace_views(const moe_shape *shape, void *ws, moe_views *views);

/* ------------------------------------------------------------------ MXFP4
 * Operands in 4 bits (OCP microscaling): a matrix [rows, cols] is cut along
 * its rows into blocks of 32 elements with one scale each.
 *   codes  [rows, cols/2] uint8: e2m1 elements (sign, then 0 0.5 1 1.5 2 3 4
 *          6), element 2i in the low nibble of byte i;
 *   scales uint8: byte s stands for 2^(s - 127), 255 for NaN, in 512-byte
 *          tiles of 128 rows x 4 blocks: the scale of (row r, block b) is byte
 *            ((r/128) * (cols/128) + b/4) * 512
 *              + (r%32) * 16 + (r%128)/32 * 4 + b%4
 *          (rows rounded up to a multiple of 128).
 * Quantisation: s = clamp(floor(log2(max|x|)) - 2 + 127, 0, 254) over the
 * block, codes = x * 2^(127-s) rounded to nearest even, saturated at 6.  A
 * block of zeros gets s = 0; a block holding a NaN or an infinity gets s = 255
 * and codes 0, so that it reads as NaN.
 * Expert weights are quantised along their reduction axis and held with that
 * axis contiguous: W [E, K, N] as the matrix [E*N, K].
 *
 * Sizes: 1 <= rows < 2^31; cols, K and N multiples of 128 from 128 to 32768;
 * 1 <= E <= 256; else MOE_ERR_UNSUPPORTED_SHAPE. */

/* Host only.  Bytes of the codes and of the scales of a [rows, cols] matrix. */
moe_status moe_mxfp4_sizes(int64_t rows, int64_t cols, size_t *code_bytes, size_t *scale_bytes);

/* Rows x [rows, cols] bf16 to codes and scales.  The scales of the rows
 * between `rows` and the next multiple of 128 are written as 0. */
moe_status moe_quantize_mxfp4(const moe_bf16 *x, int64_t rows, int64_t cols,
                              uint8_t *codes, uint8_t *scales, moe_stream_t stream);

/* Weights w [E, K, N] bf16 (K the reduction axis) to the codes and scales of
 * the matrix [E*N, K]. */
moe_status moe_quantize_weights_mxfp4(const moe_bf16 *w, int32_t E, int64_t K, int64_t N,
                                      uint8_t *codes, uint8_t *scales, moe_stream_t stream);

/* The values x [rows, cols] bf16 that codes and scales stand for (exact; past
 * bf16's range they are infinite). */
moe_status moe_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, int64_t rows,
                                int64_t cols, moe_bf16 *x, moe_stream_t stream);

/* Tokens X [T, H] bf16 quantised once each and written to their k permuted
 * rows scatter_idx [T, k]: codes and scales of the matrix [max_rows, H].
 * Padding rows are left unwritten.  ws as for the products below. */
moe_status moe_quantize_permute_mxfp4(const moe_shape *shape, const moe_bf16 *X,
                                      const int32_t *scatter_idx, uint8_t *codes, uint8_t *scales,
                                      void *ws, moe_stream_t stream);

/* The grouped gate/up product on MXFP4 operands:
 *   h[r] = bf16(silu(x_r Wg[e]) * (x_r Wu[e]))   [max_rows, I] bf16
 * for the real rows r of every expert e (rows off_pad[e] .. off_pad[e] +
 * counts[e]); padding rows of h are not written, and padding rows of the
 * operands do not reach a stored result.
 *   x_codes, x_scales: the matrix [max_rows, H] in expert order
 *   wg_*, wu_*:        the matrices [E*I, H]
 *   ws: moe_mxfp4_workspace_size bytes, or at least 256 bytes of which the
 *       first 256 were cleared (the status word and the tile counters; a
 *       product that finds its tile counter anything but cleared reports
 *       MOE_ERR_DEVICE_BOUNDS, and some of its rows may not be written)
 * The scales are applied by the tensor cores, sums are float32, h is rounded
 * once. */
moe_status moe_grouped_gemm_up_mxfp4(const moe_shape *shape, const uint8_t *x_codes,
                                     const uint8_t *x_scales, const int32_t *counts,
                                     const int32_t *off_pad, const uint8_t *wg_codes,
                                     const uint8_t *wg_scales, const uint8_t *wu_codes,
                                     const uint8_t *wu_scales, moe_bf16 *h, void *ws,
                                     moe_stream_t stream);

/* The grouped down product on MXFP4 operands: Y[r] = bf16(h_r Wd[e])
 * [max_rows, H] bf16, rows as above.
 *   h_codes, h_scales: the matrix [max_rows, I];  wd_*: the matrix [E*H, I] */
moe_status moe_grouped_gemm_down_mxfp4(const moe_shape *shape, const uint8_t *h_codes,
                                       const uint8_t *h_scales, const int32_t *counts,
                                       const int32_t *off_pad, const uint8_t *wd_codes,
                                       const uint8_t *wd_scales, moe_bf16 *Y, void *ws,
                                       moe_stream_t stream);

/* Host only.  Bytes of the workspace of moe_forward_mxfp4.  moe_workspace_init
 * clears its counters and moe_last_device_status reads its status word, as for
 * moe_forward's; moe_workspace_views does not apply to it. */
moe_status moe_mxfp4_workspace_size(const moe_shape *shape, size_t *bytes);

/* The whole layer with the experts' products in MXFP4: route, quantise and
 * permute the tokens, gate/up product with h quantised in its epilogue (to the
 * codes that quantising the bf16 h gives), down product, combine.  Weights as
 * moe_quantize_weights_mxfp4 leaves them; everything else as moe_forward. */
moe_status moe_forward_mxfp4(const moe_shape *shape, const float *logits, const moe_bf16 *X,
                             const uint8_t *wg_codes, const uint8_t *wg_scales,
                             const uint8_t *wu_codes, const uint8_t *wu_scales,
                             const uint8_t *wd_codes, const uint8_t *wd_scales, moe_bf16 *out,
                             void *ws, moe_stream_t stream);

/* --------------------------------------------------------- 8-bit integers
 * A matrix [rows, cols] in 8 bits: codes q [rows, cols] int8 and one float32
 * scale per row, s = amax / 127 with amax = max |x| of the row; it stands for
 * q s.  Quantisation: q = 127 x / amax rounded to the nearest integer, ties to
 * even (-127 .. 127), exactly.  A row of zeros gets s = 0; a row holding a NaN
 * or an infinity gets s = NaN and codes 0, so that it reads as NaN.  Expert
 * weights get a scale per output column: W [E, K, N] as the matrix [E*N, K].
 * The products also take the code -128.
 *
 * Sizes as for MXFP4. */

/* Rows x [rows, cols] bf16 to codes and scales. */
moe_status moe_quantize_int8(const moe_bf16 *x, int64_t rows, int64_t cols, int8_t *codes,
                             float *scales, moe_stream_t stream);

/* Weights w [E, K, N] bf16 (K the reduction axis) to the codes and scales of
 * the matrix [E*N, K]. */
moe_status moe_quantize_weights_int8(const moe_bf16 *w, int32_t E, int64_t K, int64_t N,
                                     int8_t *codes, float *scales, moe_stream_t stream);

/* The values bf16(q s) [rows, cols] that codes and scales stand for. */
moe_status moe_dequantize_int8(const int8_t *codes, const float *scales, int64_t rows, int64_t cols,
                               moe_bf16 *x, moe_stream_t stream);

/* Tokens X [T, H] bf16 quantised once each and written to their k permuted
 * rows scatter_idx [T, k]: codes and scales of the matrix [max_rows, H].
 * Padding rows are left unwritten.  ws as for the products below. */
moe_status moe_quantize_permute_int8(const moe_shape *shape, const moe_bf16 *X,
                                     const int32_t *scatter_idx, int8_t *codes, float *scales,
                                     void *ws, moe_stream_t stream);

/* The grouped gate/up product on 8-bit integers:
 *   h[r] = bf16(silu(g) u),  g = x_scales[r] wg_scales[n] <x_codes[r], wg_codes[n]>
 * and u alike with wu, [max_rows, I] bf16, for the real rows r of every expert;
 * padding rows as for the MXFP4 product.
 *   x_codes, x_scales: the matrix [max_rows, H] in expert order
 *   wg_*, wu_*:        the matrices [E*I, H]
 *   ws: any workspace, or at least 256 bytes whose first 256 were cleared
 * Products of codes are exact, and their float32 sums too while every partial sum
 * is below 2^24 (whatever the codes for H <= 1024).  Few rows (by the shape's T, E
 * and k) are summed in 32-bit integers, which are always exact: past 2^24 a row's
 * last bits can therefore differ between a call of few rows and one of many. */
moe_status moe_grouped_gemm_up_int8(const moe_shape *shape, const int8_t *x_codes,
                                    const float *x_scales, const int32_t *counts,
                                    const int32_t *off_pad, const int8_t *wg_codes,
                                    const float *wg_scales, const int8_t *wu_codes,
                                    const float *wu_scales, moe_bf16 *h, void *ws,
                                    moe_stream_t stream);

/* The grouped down product on 8-bit integers: Y [max_rows, H] bf16, rows as above.
 *   h_codes, h_scales: the matrix [max_rows, I];  wd_*: the matrix [E*H, I] */
moe_status moe_grouped_gemm_down_int8(const moe_shape *shape, const int8_t *h_codes,
                                      const float *h_scales, const int32_t *counts,
                                      const int32_t *off_pad, const int8_t *wd_codes,
                                      const float *wd_scales, moe_bf16 *Y, void *ws,
                                      moe_stream_t stream);

/* Host only.  Bytes of the workspace of moe_forward_int8; moe_workspace_init and
 * moe_last_device_status serve it, moe_workspace_views does not. */
moe_status moe_int8_workspace_size(const moe_shape *shape, size_t *bytes);

/* The whole layer with the experts' products on 8-bit integers: route, quantise
 * and permute the tokens, gate/up product, h quantised row by row, down product,
 * combine.  Weights as moe_quantize_weights_int8 leaves them; everything else as
 * moe_forward. */
moe_status moe_forward_int8(const moe_shape *shape, const float *logits, const moe_bf16 *X,
                            const int8_t *wg_codes, const float *wg_scales, const int8_t *wu_codes,
                            const float *wu_scales, const int8_t *wd_codes, const float *wd_scales,
                            moe_bf16 *out, void *ws, moe_stream_t stream);

/* ----------------------------------------------------------- balance loss
 * A token takes part when its mask byte is non-zero (or mask is NULL) and not
 * all of its logits are -inf; n tokens do.  With p = softmax(logits) over
 * them:
 *   counts[e]     = picks (t, j) with topk_ids[t, j] = e
 *   mean_probs[e] = sum_t p[t, e] / n
 *   losses[0]     = E * sum_e counts[e]/(n k) * mean_probs[e]   (balance)
 *   losses[1]     = sum_t logsumexp(logits[t])^2 / n            (z-loss)
 * and all of them are 0 for n = 0.  A NaN or +inf logit of a token that takes
 * part makes the losses NaN; tokens that take no part are not looked at. */

/* Host only.  Bytes of the workspace of moe_balance_loss (at most 1 MiB). */
moe_status moe_balance_workspace_size(const moe_shape *shape, size_t *bytes);

/*   logits     [T, E] float32 (-inf allowed), topk_ids [T, k] int32 (moe_route's)
 *   mask       [T] bytes or NULL
 *   counts     [E] int32 out, num_tokens [1] int32 out (n)
 *   mean_probs [E] float32 out, losses [2] float32 out
 *   ws         moe_balance_workspace_size bytes, the first 256 cleared once
 *              (moe_workspace_init); an expert id out of range is not counted
 *              and reported by moe_last_device_status, as is a counter that
 *              was not cleared (the results may then be stale)
 * H and I of the shape are not used. */
moe_status moe_balance_loss(const moe_shape *shape, const float *logits, const int32_t *topk_ids,
                            const uint8_t *mask, int32_t *counts, int32_t *num_tokens,
                            float *mean_probs, float *losses, void *ws, moe_stream_t stream);

/* The gradient to the logits, counts held constant:
 *   dlogits[t, e] = p[t, e] * ( g0 E/n (f[e] - sum_j f[j] p[t, j])
 *                             + g1 2/n logsumexp(logits[t]) ),  f = counts/(n k)
 * and 0 for tokens that take no part.
 *   counts, num_tokens: moe_balance_loss's; grad_losses [2] float32 (g0, g1),
 *   the gradients of the two losses; dlogits [T, E] float32 out */
moe_status moe_balance_loss_backward(const moe_shape *shape, const float *logits,
                                     const uint8_t *mask, const int32_t *counts,
                                     const int32_t *num_tokens, const float *grad_losses,
                                     float *dlogits, moe_stream_t stream);

/* --------------------------------------------------------------- training
 * The backward pass of the experts' gated feed-forward and of the layer around
 * it.  Per expert, over its rows,
 *   g = x Wg, u = x Wu, s = sigmoid(g), h = g s u, Y = h Wd
 *   dh = dY Wd^T, dg = dh u s (1 + g (1 - s)), du = dh g s
 *   dx = dg Wg^T + du Wu^T, dWg = x^T dg, dWu = x^T du, dWd = h^T dY
 * with float32 sums, and g, u, h, dg, du and every result rounded once to bf16.
 * One expert that takes every token (E = k = 1, counts[0] = T, off_pad = {0, T rounded
 * up to 128}) is a dense gated feed-forward.
 *
 * Buffers in expert order have max_rows rows, as above; padding rows are not
 * written, and what they hold does not reach a result.  ws: any workspace, or
 * at least 256 bytes whose first 256 were cleared (the status word and the tile
 * counters; a product that finds its counter anything but cleared reports
 * MOE_ERR_DEVICE_BOUNDS).  Outputs may not overlap inputs or one another. */

/* moe_grouped_gemm_up_rows that also keeps g and u, [max_rows, I] bf16 (h is
 * formed from the float32 sums: the same bits). */
moe_status moe_grouped_gemm_up_train(const moe_shape *shape, const moe_bf16 *Xp,
                                     const int32_t *counts, const int32_t *off_pad,
                                     const moe_bf16 *W_gate, const moe_bf16 *W_up, moe_bf16 *g,
                                     moe_bf16 *u, moe_bf16 *h, void *ws, moe_stream_t stream);

/* Gradients of the combine and of the routing weights:
 *   dY[row(t, j)] = topk_w[t, j] dout[t]                     [max_rows, H] bf16
 *   dlogits[t, e] = sum over j with topk_ids[t, j] = e of
 *                   w_j (dw_j - sum_l w_l dw_l),  dw_j = <dout[t], Y[row(t, j)]>
 * [T, E] float32 (zero where nothing was picked), which is the gradient of the
 * softmax, top-k and renormalisation with the picks held.  A row or an id out of
 * range takes no part and is reported.
 *   Y, scatter_idx, topk_ids, topk_w: the forward's; dout [T, H] bf16 */
moe_status moe_combine_backward(const moe_shape *shape, const moe_bf16 *Y,
                                const int32_t *scatter_idx, const int32_t *topk_ids,
                                const float *topk_w, const moe_bf16 *dout, moe_bf16 *dY,
                                float *dlogits, void *ws, moe_stream_t stream);

/* dg and du [max_rows, I] from dY [max_rows, H]; the activation's derivative is
 * formed in the product's epilogue, from the float32 dh. */
moe_status moe_grouped_gemm_down_backward(const moe_shape *shape, const moe_bf16 *dY,
                                          const int32_t *counts, const int32_t *off_pad,
                                          const moe_bf16 *W_down, const moe_bf16 *g,
                                          const moe_bf16 *u, moe_bf16 *dg, moe_bf16 *du, void *ws,
                                          moe_stream_t stream);

/* dXp [max_rows, H] from dg and du: both products in one sum. */
moe_status moe_grouped_gemm_up_backward(const moe_shape *shape, const moe_bf16 *dg,
                                        const moe_bf16 *du, const int32_t *counts,
                                        const int32_t *off_pad, const moe_bf16 *W_gate,
                                        const moe_bf16 *W_up, moe_bf16 *dXp, void *ws,
                                        moe_stream_t stream);

/* The gradients of the three weights, [E, H, I], [E, H, I] and [E, I, H] bf16,
 * from the rows and their gradients; zero for an expert without rows. */
moe_status moe_grouped_gemm_weight_backward(const moe_shape *shape, const moe_bf16 *Xp,
                                            const moe_bf16 *h, const moe_bf16 *dg,
                                            const moe_bf16 *du, const moe_bf16 *dY,
                                            const int32_t *counts, const int32_t *off_pad,
                                            moe_bf16 *dW_gate, moe_bf16 *dW_up, moe_bf16 *dW_down,
                                            void *ws, moe_stream_t stream);

/* The gradient of the row gather: dX[t] = bf16(sum_j dXp[scatter_idx[t, j]]),
 * a float32 sum in slot order. */
moe_status moe_permute_backward(const moe_shape *shape, const moe_bf16 *dXp,
                                const int32_t *scatter_idx, moe_bf16 *dX, void *ws,
                                moe_stream_t stream);

/* moe_forward (the same output, bit for bit) that keeps g and u [max_rows, I]
 * for the backward pass, which also reads the routing, Xp, h and Y left in
 * `ws`: one workspace per layer whose backward pass is still to come. */
moe_status moe_forward_train(const moe_shape *shape, const float *logits, const moe_bf16 *X,
                             const moe_bf16 *W_gate, const moe_bf16 *W_up, const moe_bf16 *W_down,
                             moe_bf16 *g, moe_bf16 *u, moe_bf16 *out, void *ws,
                             moe_stream_t stream);

/* Host only.  Bytes of the scratch of moe_backward, which layers may share;
 * moe_workspace_init clears its counters and moe_last_device_status reads its
 * status word. */
moe_status moe_backward_workspace_size(const moe_shape *shape, size_t *bytes);

/* The layer's backward pass: dout [T, H] bf16 to dX [T, H], the gradients of
 * the three weights, and dlogits [T, E] float32 (of the routing weights alone:
 * moe_balance_loss_backward's adds to it).
 *   g, u, ws: as moe_forward_train left them (read, not changed)
 *   bws:      moe_backward_workspace_size bytes */
moe_status moe_backward(const moe_shape *shape, const moe_bf16 *W_gate, const moe_bf16 *W_up,
                        const moe_bf16 *W_down, const moe_bf16 *g, const moe_bf16 *u,
                        const moe_bf16 *dout, moe_bf16 *dX, moe_bf16 *dW_gate, moe_bf16 *dW_up,
                        moe_bf16 *dW_down, float *dlogits, const void *ws, void *bws,
                        moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_H */
