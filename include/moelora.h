/*
 * moelora.h -- C ABI of the fused MoE expert-FFN layer with multi-LoRA for
 * AMD Instinct MI355X (gfx950).
 *
 * What the layer computes follows the AWS Machine Learning blog post
 * "Efficiently serve dozens of fine-tuned models with vLLM on Amazon
 * SageMaker AI and Amazon Bedrock" ([AWS] below), section "Implementing
 * multi-LoRA inference for MoE models in vLLM" and its Figure 1: a router
 * sends each token to its top-k experts; each expert applies a gate_up
 * projection and a down projection; a LoRA adapter on a projection with base
 * weight W adds x A B (shrink z = x A to rank r, expand z B back), and every
 * token carries its own adapter id, or none.  For each routed (token, expert)
 * pair with adapter a (a = -1: none):
 *
 *     g   = x W_gu[e]^T + [a >= 0] (x A_gu[a][e]^T) B_gu[a][e]^T   (width 2I)
 *     h   = SiLU(g[0:I]) * g[I:2I],   SiLU(v) = v / (1 + exp(-v))
 *     y   = h W_d[e]^T  + [a >= 0] (h A_d[a][e]^T) B_d[a][e]^T     (width H)
 *     out[t] = sum_j w[t][j] * y(t, ids[t][j])
 *
 * The router, when used, keeps the k largest logits (ties to the lower
 * expert index, listed largest first) and sets w = softmax over the kept
 * logits (softmax over all E followed by renormalisation over the kept k).
 * Logits are expected to be finite: a NaN's place in the order is
 * unspecified (the picks are still k distinct experts in range).
 * The post fixes neither the router formula, the activation nor the gate/up
 * split; these are the readings used here.
 *
 * Storage: row-major, contraction dimension contiguous, elements of the
 * layer dtype (float32, or bf16 as 16-bit patterns):
 *     x        [T][H]          out      [T][H]
 *     W_gu     [E][2I][H]      rows 0..I-1 gate, I..2I-1 up
 *     W_d      [E][H][I]
 *     A_gu     [NA][E][r][H]   B_gu     [NA][E][2I][r]
 *     A_d      [NA][E][r][I]   B_d      [NA][E][H][r]
 *     router_logits [T][E] float32;  topk_ids [T][k] int32;
 *     topk_w [T][k] float32;  adapter_ids [T] int32 (-1 = none)
 * Every device pointer must be 16-byte aligned; the workspace 256-byte
 * aligned.
 *
 * Ownership: the caller allocates and owns every device buffer, the
 * workspace and the stream.  The library owns only the plan (a host
 * object).  moelora_forward only enqueues kernels on the given stream: it
 * never synchronises or allocates, so it can be captured in a HIP graph, and
 * nothing is specialised on the token count.  Kernels are compiled ahead of
 * time; the HIP runtime loads their code on first use, so the first forward
 * of a plan on a device (the current device) looks up every kernel that
 * plan can launch at any token count up to max_tokens, and no later forward
 * loads code ([AWS] "Execution optimizations": loading code for each new
 * context length cost a tenfold time-to-first-token regression).
 *
 * Errors: every entry point returns a status; nothing throws or aborts
 * across the ABI.  Device-resident ids are preconditions: expert ids in
 * [0, E), adapter ids in [-1, NA).  A row with an out-of-range expert id is
 * dropped (adds nothing to its token's output) and an out-of-range adapter
 * id counts as -1; either sets a bit in the device error word that
 * moelora_read_device_error returns.  No kernel reads or writes out of
 * bounds on bad ids.
 */
#ifndef MOELORA_H
#define MOELORA_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__) || defined(__clang__)
#define MOELORA_API __attribute__((visibility("default")))
#else
#define MOELORA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum moelora_status {
    MOELORA_OK = 0,
    MOELORA_ERR_INVALID_ARG = -1,  /* null / misaligned pointer, bad size  */
    MOELORA_ERR_UNSUPPORTED = -2,  /* shape or dtype outside the limits    */
    MOELORA_ERR_WORKSPACE = -3,    /* workspace too small                  */
    MOELORA_ERR_HIP = -4,          /* a HIP runtime call or launch failed  */
    MOELORA_ERR_DEVICE = -5,       /* the device error word is non-zero    */
    MOELORA_ERR_TOO_LARGE = -6     /* beyond moelora_forward_noalloc's
                                      static scratch buffer                */
} moelora_status;

/* Element types.  MOELORA_BF16_FP8W: x, out and the LoRA weights bf16; the
 * base weights W_gu and W_d one byte per element, an OCP 8-bit floating-point
 * E4M3 code, with one float32 scale per weight row: the weight is
 * scale[row] times the code's value (the aib.vote news item on SageMaker
 * fused-MoE kernel optimizations, second item, routes FP8 MoE layers to a
 * fused path; it gives no quantisation scheme, and one scale per output row
 * is the reading taken here).  Each of w_gate_up / w_down then points at the
 * codes, [E][2I] rows of H codes / [E][H] rows of I codes, each row padded
 * with zero bytes to a multiple of 128 bytes (row pitch P = round_up(H, 128)
 * / round_up(I, 128), so every row starts on a 128-byte line), followed at
 * the next 256-byte boundary (byte offset round_up(E*2I*P, 256) /
 * round_up(E*H*P, 256)) by the scales, float32 [E][2I] / [E][H].  Requires H
 * and I multiples of 64 and r a multiple of 8. */
typedef enum moelora_dtype {
    MOELORA_F32 = 0,
    MOELORA_BF16 = 1,
    MOELORA_BF16_FP8W = 2
} moelora_dtype;

/* Bits of the device error word. */
#define MOELORA_DEVERR_EXPERT_ID 1   /* an expert id outside [0, E)        */
#define MOELORA_DEVERR_ADAPTER_ID 2  /* an adapter id outside [-1, NA)     */

/* Shape of one layer.  Limits (else MOELORA_ERR_UNSUPPORTED):
 * 1 <= E <= 1024, E * (NA + 1) <= 8448, 1 <= k <= min(E, 32),
 * 0 <= NA, 0 <= r <= 256 (r >= 1 when NA >= 1), 1 <= H, I <= 65536,
 * 0 <= max_tokens, max_tokens * k <= 2^24; flags: a combination of the
 * MOELORA_FLAG_* bits below (any other bit: MOELORA_ERR_UNSUPPORTED). */
typedef struct moelora_desc {
    int32_t max_tokens;
    int32_t hidden;      /* H */
    int32_t inter;       /* I (gate_up produces 2I) */
    int32_t n_experts;   /* E */
    int32_t top_k;       /* k */
    int32_t n_adapters;  /* NA */
    int32_t rank;        /* r */
    int32_t dtype;       /* moelora_dtype */
    uint32_t flags;      /* MOELORA_FLAG_* bits */
} moelora_desc;

/* Flags.  Both behaviours are always on in this library, so the bits are
 * accepted and change nothing; they exist so a caller can state that it
 * relies on them.
 *   DETERMINISTIC    results are bitwise repeatable for a given plan, input
 *                    and token count: split contractions (the split-K shrink
 *                    of [AWS] "Kernel optimizations", the split down GEMM)
 *                    write separate fp32 partials that their consumer adds
 *                    in a fixed order; no kernel uses floating-point atomics.
 *   DEBUG_CHECK_IDS  device-resident ids are range-checked: an expert id
 *                    outside [0, E) drops its row, an adapter id outside
 *                    [-1, NA) counts as -1, and either sets a bit of the
 *                    device error word (moelora_read_device_error). */
#define MOELORA_FLAG_DETERMINISTIC 1u
#define MOELORA_FLAG_DEBUG_CHECK_IDS 2u

typedef struct moelora_plan_s *moelora_plan_t;
typedef struct ihipStream_t *moelora_stream_t; /* the same type as hipStream_t */

/* Validate the shape and choose kernels, block size and split-K for every
 * token count up to max_tokens.  Host only: no device memory is touched and
 * no code is compiled or loaded; every kernel is compiled ahead of time and
 * takes the token count as a run-time argument, and the choices are made
 * here, once, for all token counts, because [AWS] "Execution optimizations"
 * traces a tenfold time-to-first-token regression to kernels recompiled for
 * each new context length.  Tuning switches in the environment (MOELORA_*)
 * are read here and never by a forward.  *workspace_bytes receives the
 * largest workspace any forward of 0..max_tokens tokens needs (every token
 * count is checked).  On success *plan must later be released with
 * moelora_plan_destroy.  Errors: MOELORA_ERR_INVALID_ARG for null
 * pointers, MOELORA_ERR_UNSUPPORTED for a shape, dtype or flag outside the
 * limits above. */
MOELORA_API moelora_status moelora_plan(const moelora_desc *desc, moelora_plan_t *plan,
                            size_t *workspace_bytes);

MOELORA_API void moelora_plan_destroy(moelora_plan_t plan);

/* Enqueue one layer call on `stream` (NULL = the null stream).
 *   n_tokens       0 <= n_tokens <= max_tokens; 0 is a no-op
 *   x              [T][H] layer dtype
 *   router_logits  [T][E] float32; NULL exactly when topk_ids and topk_w
 *                  are given
 *   topk_ids       [T][k] int32, or NULL to route from the logits
 *   topk_w         [T][k] float32, or NULL (with topk_ids NULL)
 *   adapter_ids    [T] int32, or NULL: no adapter for any token
 *   w_gate_up, w_down   base expert weights (required)
 *   lora_a_gu, lora_b_gu, lora_a_d, lora_b_d   adapter weights; all four
 *                  NULL (or NA == 0, or adapter_ids NULL) skips every LoRA
 *                  kernel ([AWS] "Execution optimizations": layers without
 *                  adapters exit early); otherwise all four are required
 *   out            [T][H] layer dtype, written (not accumulated)
 *   workspace      >= the size moelora_plan returned, 256-byte aligned; its
 *                  contents need no initialisation.  Concurrent forwards
 *                  need distinct workspaces.
 * The call returns after enqueueing; results are ready when the stream
 * reaches that point. */
MOELORA_API moelora_status moelora_forward(moelora_plan_t plan, int32_t n_tokens,
                               const void *x, const float *router_logits,
                               const int32_t *topk_ids, const float *topk_w,
                               const int32_t *adapter_ids,
                               const void *w_gate_up, const void *w_down,
                               const void *lora_a_gu, const void *lora_b_gu,
                               const void *lora_a_d, const void *lora_b_d,
                               void *out, void *workspace,
                               size_t workspace_bytes,
                               moelora_stream_t stream);

/* moelora_forward for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * allocation.  Same arguments and results as moelora_forward, without the
 * workspace: the call uses a static device array of the library,
 * MOELORA_STATIC_SCRATCH_BYTES (64 MiB) per GPU, allocated with the
 * library's code on each GPU it runs on and held until the process ends.
 * The call allocates nothing; its first call on a GPU looks up that GPU's
 * copy of the array.  `stream` must belong to the current device
 * (else MOELORA_ERR_INVALID_ARG).  A call whose workspace (the size
 * moelora_plan_info reports for n_tokens) exceeds the array returns
 * MOELORA_ERR_TOO_LARGE before touching the device.  Every call on a GPU
 * shares that GPU's array: calls that overlap on one GPU (two streams, two
 * threads) race and must be serialised by the caller, e.g. on one stream.
 * The array's contents need no initialisation; moelora_read_device_error
 * does not apply (its error word lives in the array). */
#define MOELORA_STATIC_SCRATCH_BYTES ((size_t)64 << 20)
MOELORA_API moelora_status moelora_forward_noalloc(moelora_plan_t plan, int32_t n_tokens,
                               const void *x, const float *router_logits,
                               const int32_t *topk_ids, const float *topk_w,
                               const int32_t *adapter_ids,
                               const void *w_gate_up, const void *w_down,
                               const void *lora_a_gu, const void *lora_b_gu,
                               const void *lora_a_d, const void *lora_b_d,
                               void *out, moelora_stream_t stream);

/* ---------------------------------------------------------------------
 * Stand-alone operators: the layer's steps for callers that put their own
 * expert function, gradients or block-scaled FP8 weights between them.
 *
 * Common rules.  Row-major, contiguous; every device pointer 16-byte
 * aligned and on the current device; each call enqueues on `stream`,
 * allocates nothing, synchronises nothing and keeps nothing, so it can be
 * captured in a HIP graph.  Inputs and outputs must not overlap.  Results
 * repeat bit for bit (no floating-point atomics), sums run in float32 and are
 * rounded once.  dtype is MOELORA_F32 or MOELORA_BF16 (else
 * MOELORA_ERR_UNSUPPORTED).  The first call on a device loads the code of
 * all of these operators.
 *
 * Token order.  T tokens, k experts each, R = T k routed rows p = t k + j.
 * Limits (else MOELORA_ERR_UNSUPPORTED): 1 <= hidden <= 65536, 1 <= E <=
 * 1024, 1 <= k <= 32, R <= 2^24.  k may exceed E: a shard that holds some of
 * the experts numbers those 0 .. E-1 and marks rows of the others with any
 * id outside [0, E) (say -1); such rows are dropped.
 *
 * moelora_dispatch sorts the routed rows by expert, stably (ascending p
 * inside an expert), and copies their tokens into that order:
 *   expert_start [E+1]  first sorted position of each expert's rows;
 *                       expert_start[E] = rows kept
 *   sorted_rows  [R]    routed row p at each sorted position, R past the
 *                       rows kept
 *   row_pos      [T][k] sorted position of each routed row, -1 if dropped
 *   xs           [R][H] x[sorted_rows[pos] / k]; rows past the rows kept
 *                       are left as they were.  NULL (x may be NULL
 *                       too): the order only.
 * workspace: moelora_dispatch_workspace bytes (0 for small batches, at
 * most 1024 E; enough for every smaller n_tokens of the same n_experts and
 * top_k too), no initialisation; calls that overlap need one each.
 * n_tokens = 0 writes expert_start (zeros) and reads nothing. */
MOELORA_API moelora_status moelora_dispatch_workspace(int32_t n_tokens, int32_t n_experts,
                               int32_t top_k, size_t *workspace_bytes);
MOELORA_API moelora_status moelora_dispatch(int32_t n_tokens, int32_t hidden, int32_t n_experts,
                               int32_t top_k, int32_t dtype, const void *x,
                               const int32_t *topk_ids, int32_t *expert_start,
                               int32_t *sorted_rows, int32_t *row_pos, void *xs,
                               void *workspace, size_t workspace_bytes,
                               moelora_stream_t stream);

/* Gradient of the copy: dx[t] = sum_j dxs[row_pos[t][j]], ascending j; a
 * dropped row adds nothing.  row_pos entries outside [0, R) count as
 * dropped here and in the calls below.  dxs [R][H], dx [T][H]. */
MOELORA_API moelora_status moelora_dispatch_backward(int32_t n_tokens, int32_t hidden,
                               int32_t top_k, int32_t dtype, const void *dxs,
                               const int32_t *row_pos, void *dx,
                               moelora_stream_t stream);

/* out[t] = sum_j topk_w[t][j] ys[row_pos[t][j]], ascending j.  ys [R][H],
 * topk_w [T][k] float32, out [T][H] (zeros where every row was dropped). */
MOELORA_API moelora_status moelora_combine(int32_t n_tokens, int32_t hidden, int32_t top_k,
                               int32_t dtype, const void *ys, const int32_t *row_pos,
                               const float *topk_w, void *out, moelora_stream_t stream);

/* Gradients of moelora_combine, given dout [T][H]:
 *   dys [R][H]  dys[row_pos[t][j]] = topk_w[t][j] dout[t]; rows that no
 *               routed row points to are left as they were.  Positions in
 *               [0, R) must differ (those of moelora_dispatch do): of a row
 *               pointed to twice one of the writes stays, not their sum.
 *               NULL: not wanted (topk_w may then be NULL).
 *   dw [T][k]   float32, <dout[t], ys[row_pos[t][j]]>, 0 for a dropped row.
 *               NULL: not wanted (ys may then be NULL).  */
MOELORA_API moelora_status moelora_combine_backward(int32_t n_tokens, int32_t hidden,
                               int32_t top_k, int32_t dtype, const void *dout,
                               const void *ys, const int32_t *row_pos,
                               const float *topk_w, void *dys, float *dw,
                               moelora_stream_t stream);

/* Block-scaled E4M3.  A row of `width` = K elements is stored as one code a
 * byte, padded with zero bytes to the pitch P = round_up(K, 128), and one
 * float32 scale per block of 128: value = scale * code.  KB = P / 128.
 *   rows     codes [M][P], scales [KB][M] (block-major)
 *   weights  codes [mats][N][P], scales [mats][NB][KB], one per 128 x 128
 *            block, NB = ceil(N / 128)
 * The quantisers choose the smallest power of two 2^e >= max|v| / 448 (e >=
 * -126) of the block's finite elements as its scale and round v / 2^e, which
 * is exact, to the nearest code, ties to even; an element that is not finite
 * gets the NaN code.  The product takes any float32 scales; a block whose two
 * scales multiply to less than 2^-126 may be off by 2^-125.
 * Limits (else MOELORA_ERR_UNSUPPORTED): 1 <= K <= 65536, rows of x <=
 * 2^24, 1 <= N <= 131072, mats <= 65535, E <= 1024. */

/* Rows r of x (rows = NULL; then n_src >= n_rows and row_div = 1), or rows
 * rows[r] / row_div of the n_src rows of x: with the sorted_rows of
 * moelora_dispatch and row_div = k the tokens in expert order.  Where
 * rows[r] is negative or points past n_src (the tail of sorted_rows does),
 * row r of codes and scales is left as it was. */
MOELORA_API moelora_status moelora_quantize_rows(int32_t n_rows, int32_t width, int32_t dtype,
                               const void *x, int32_t n_src, const int32_t *rows,
                               int32_t row_div, void *codes, float *scales,
                               moelora_stream_t stream);

/* Weights w [mats][N][K].  codes_t, scales_t (both or neither): the same
 * codes transposed, [mats][K][round_up(N, 128)] and [mats][KB][NB], the
 * weights of the product's gradient in its rows: with dy [M][N] quantised by
 * rows, dx = moelora_fp8_gemm of dy and (codes_t, scales_t), n_out = K,
 * width = N. */
MOELORA_API moelora_status moelora_quantize_weights(int32_t n_mats, int32_t rows,
                               int32_t width, int32_t dtype, const void *w, void *codes,
                               float *scales, void *codes_t, float *scales_t,
                               moelora_stream_t stream);

/* The grouped product: for the rows m of expert e, expert_start[e] <= m <
 * expert_start[e+1],
 *   out[m][n] = sum_b scales[b][m] w_scales[e][n/128][b]
 *               sum_{k in block b} codes[m][k] w_codes[e][n][k]
 * in float32, rounded once to out_dtype (MOELORA_F32, MOELORA_BF16), out
 * [M][N].  For MOELORA_F32 the products are exact and summed in float32.  For
 * MOELORA_BF16 the FP8 matrix core forms the sums over a block, except where
 * rows are few: they are off by at most 7 2^-13 of the block's sum of
 * magnitudes (on normal data 1.5e-5 of the result).  Rows outside every expert's range are left as they were.
 * expert_start = NULL with n_experts = 1: all rows (a dense product).
 * Entries of expert_start are clamped into [0, M]; they must not fall.
 * With MOELORA_FP8_SILU_MUL the weights of an expert are two matrices, gate
 * then up (w_codes [E][2][N][P], w_scales [E][2][NB][KB]: mats = 2 E), and
 * out = SiLU(gate) * up: for MOELORA_F32 within 2^-18 of the value that the
 * float32 gate and up give (and steps of the smallest subnormal), with
 * sigmoids below 2^-251 as zero; for MOELORA_BF16 (before the rounding) within
 * (|gate| + 4) 2^-23 of it, with sigmoids below 2^-126 as zero. */
#define MOELORA_FP8_SILU_MUL 1u
MOELORA_API moelora_status moelora_fp8_gemm(int32_t n_rows, int32_t n_out, int32_t width,
                               int32_t n_experts, int32_t out_dtype, uint32_t flags,
                               const void *codes, const float *scales,
                               const int32_t *expert_start, const void *w_codes,
                               const float *w_scales, void *out, moelora_stream_t stream);

/* A one-line description of the kernel that a product of these sizes takes
 * (for logs; host only): NUL-terminated, truncated to buf_len. */
MOELORA_API moelora_status moelora_fp8_gemm_info(int32_t n_rows, int32_t n_out, int32_t width,
                               int32_t n_experts, int32_t out_dtype, uint32_t flags,
                               char *buf, size_t buf_len);

/* The router by itself, its losses and their gradient.  logits [T][E] of
 * dtype; token_mask [T] one byte a token, 0: the token is padding (NULL: no
 * token is).  An expert is available to a token that is no padding if its logit
 * is above -inf and not NaN (so -inf switches an expert off); a token with none
 * counts like padding.  p[t] is the softmax over the available experts, lse[t]
 * the logarithm of its sum (probabilities below 2^-126 of the largest count as
 * zero; of several logits of +inf each has the same share).
 * Limits (else MOELORA_ERR_UNSUPPORTED): 1 <= E <= 1024, 1 <= k <= min(E, 32),
 * T k <= 2^24.
 *
 * moelora_route: the k largest available logits of each token, largest first,
 * ties to the lower expert index:
 *   topk_ids [T][k]  -1 where no expert is left (moelora_dispatch drops those)
 *   topk_w   [T][k]  float32, the softmax over the picked logits, or, with
 *                    MOELORA_ROUTE_SOFTMAX_ALL, their p; 0 for an id of -1 */
#define MOELORA_ROUTE_SOFTMAX_ALL 1u
MOELORA_API moelora_status moelora_route(int32_t n_tokens, int32_t n_experts, int32_t top_k,
                               int32_t dtype, uint32_t flags, const void *logits,
                               const uint8_t *token_mask, int32_t *topk_ids, float *topk_w,
                               moelora_stream_t stream);

/* Per-expert counts and the router's losses over the n tokens that are no
 * padding:
 *   counts   [E+1]  picks of each expert (ids outside [0, E) and those of
 *                   padding do not count); counts[E] = n
 *   prob_sum [E]    float32, sum over the tokens of p[t][e]
 *   loss     [2]    float32, E / (k n^2) sum_e counts[e] prob_sum[e] (1 where
 *                   the experts are used alike) and sum_t lse[t]^2 / n; zeros
 *                   where n = 0
 * All are written whole, also for n_tokens = 0, which reads nothing.
 * workspace: moelora_balance_loss_workspace bytes (0 for small batches, at
 * most 4096 (E + 2); enough for every smaller n_tokens of the same n_experts
 * and top_k too), no initialisation; calls that overlap need one each. */
MOELORA_API moelora_status moelora_balance_loss_workspace(int32_t n_tokens, int32_t n_experts,
                               int32_t top_k, size_t *workspace_bytes);
MOELORA_API moelora_status moelora_balance_loss(int32_t n_tokens, int32_t n_experts, int32_t top_k,
                               int32_t dtype, const void *logits, const uint8_t *token_mask,
                               const int32_t *topk_ids, int32_t *counts, float *prob_sum,
                               float *loss, void *workspace, size_t workspace_bytes,
                               moelora_stream_t stream);

/* The gradient in the logits of the routing weights, of both losses, or of all
 * three in one pass: dlogits [T][E] of dtype, written whole (zeros for padding
 * and where an expert is not available).
 *   dtopk_w [T][k]  float32, the gradient of topk_w (moelora_combine_backward
 *                   makes it); needs topk_ids and topk_w as moelora_route gave
 *                   them with the same flags.  Ids outside [0, E) add nothing.
 *                   NULL: not wanted (topk_ids and topk_w may then be NULL).
 *   counts [E+1], dloss [2]  of moelora_balance_loss, and the float32 gradients
 *                   of its two losses.  Counts are constants of the gradient.
 *                   Summed over several devices, the counts (and, for the
 *                   loss itself, prob_sum) give the gradient of the loss over
 *                   all of their tokens.  NULL (both): not wanted. */
MOELORA_API moelora_status moelora_route_backward(int32_t n_tokens, int32_t n_experts,
                               int32_t top_k, int32_t dtype, uint32_t flags, const void *logits,
                               const uint8_t *token_mask, const int32_t *topk_ids,
                               const float *topk_w, const float *dtopk_w, const int32_t *counts,
                               const float *dloss, void *dlogits, moelora_stream_t stream);

/* 4-bit weights.  A weight is an E2M1 code (bit 3 the sign; 0, 0.5, 1, 1.5, 2,
 * 3, 4, 6) times 2^(s - 127), s a byte that the 32 weights of a group along K
 * share (255: NaN).  A matrix [N][K] is kept in tiles of 16 rows x 128 columns,
 * NT = ceil(N / 16), KB = ceil(K / 128), KQ = ceil(KB / 4), zeros past N and K:
 *   codes   [mats][NT][KB][64][16] bytes; of tile (i, j), entry 16 g + r holds
 *           row 16 i + r, columns 128 j + 32 g .. + 31, two codes a byte, the
 *           lower column in the low half
 *   scales  [mats][NT][KQ][64][4] bytes; entry 16 g + r of (i, q) holds the
 *           scales of that group in tiles 4 q .. 4 q + 3
 * (1024 mats NT KB bytes and 256 mats NT KQ).
 * Limits (else MOELORA_ERR_UNSUPPORTED): 1 <= N <= 131072, 1 <= K <= 65536,
 * mats <= 65535, mats NT KQ <= 2^26 - 4.
 *
 * From weights w [mats][N][K] of dtype: the scale of a group is the smallest
 * power of two 2^e >= max|w| / 6 (e >= -125), and w / 2^e, which is exact, is
 * rounded to the nearest code, ties to even (from 1.75 2^127 on, where that is
 * 2^128, to the code below).  A group with an element that is not finite gets
 * the NaN scale and zero codes. */
MOELORA_API moelora_status moelora_quantize_weights_fp4(int32_t n_mats, int32_t rows,
                               int32_t width, int32_t dtype, const void *w, void *codes,
                               void *scales, moelora_stream_t stream);

/* From a checkpoint's row-major form: row_codes [mats][N][ceil(K / 2)] bytes,
 * two codes each, the lower column in the low half, and row_scales
 * [mats][N][ceil(K / 32)] bytes. */
MOELORA_API moelora_status moelora_pack_weights_fp4(int32_t n_mats, int32_t rows, int32_t width,
                               const void *row_codes, const void *row_scales, void *codes,
                               void *scales, moelora_stream_t stream);

/* The values w [mats][N][K] that codes and scales stand for.  Both dtypes hold
 * them exactly (from 2^128 on they are infinite). */
MOELORA_API moelora_status moelora_dequantize_weights_fp4(int32_t n_mats, int32_t rows,
                               int32_t width, int32_t dtype, const void *codes,
                               const void *scales, void *w, moelora_stream_t stream);

/* The grouped product on 4-bit weights: for the rows m of expert e,
 * expert_start[e] <= m < expert_start[e+1],
 *   out[m][n] = sum_k x[m][k] w[e][n][k]
 * with x [M][K] and out [M][N] of dtype; products are exact, summed in float32
 * and rounded once (of float32 rows the products of three parts of eight
 * significant bits each, the last a multiple of 2^-133: an element below 2^-110
 * counts as cut to such a multiple; whole where K < 4).  Rows outside every
 * expert's range are left as they were.
 * expert_start = NULL with n_experts = 1: all rows (a dense product).
 * Entries of expert_start are clamped into [0, M]; they must not fall.
 * With MOELORA_FP4_SILU_MUL the weights of an expert are two matrices, gate
 * then up (mats = 2 E), and out = SiLU(gate) * up, in float32 as of
 * moelora_fp8_gemm.  Limits: those of the weights and M <= 2^24, M N <= 2^34,
 * E <= 1024. */
#define MOELORA_FP4_SILU_MUL 1u
MOELORA_API moelora_status moelora_fp4_gemm(int32_t n_rows, int32_t n_out, int32_t width,
                               int32_t n_experts, int32_t dtype, uint32_t flags, const void *x,
                               const int32_t *expert_start, const void *w_codes,
                               const void *w_scales, void *out, moelora_stream_t stream);

/* A one-line description of the kernel that a product of these sizes takes
 * (for logs; host only): NUL-terminated, truncated to buf_len. */
MOELORA_API moelora_status moelora_fp4_gemm_info(int32_t n_rows, int32_t n_out, int32_t width,
                               int32_t n_experts, int32_t dtype, uint32_t flags,
                               char *buf, size_t buf_len);

MOELORA_API const char *moelora_status_string(moelora_status status);

/* ---------------------------------------------------------------------
 * Inspection hooks (tests and benchmarks).
 *
 * Alignment: the rows p = t*k + j are grouped per expert, each group padded
 * to a multiple of the block size BM (one BM shared by the four LoRA ops and
 * the base GEMMs, [AWS] "Tuning kernel configurations for Amazon SageMaker
 * AI and Amazon Bedrock"), and inside a group ordered by adapter (base-only
 * rows last), then by p ([AWS] "Implementing multi-LoRA inference for MoE
 * models in vLLM": expert routing compounded with adapter selection).  After
 * a forward of n_tokens tokens the workspace holds, at the offsets below
 * (bytes from the workspace start, int32 arrays):
 *   topk_ids [R], topk_w [R] (float32)  the router's output (only when the
 *                  forward routed from logits)
 *   sorted_rows [cap]       rows per expert; sentinel R in padding and after
 *                           num_padded
 *   block_expert [nblk]     expert of each block, -1 past num_padded
 *   seg_start [E+1]         padded start of each expert's rows
 *   lora_seg [max_seg][4]   (expert, adapter, start, len) for every run of
 *                           rows sharing an expert and an adapter >= 0, in
 *                           (expert, adapter) order; unused (-1, -1, 0, 0)
 *   tiles [max_tiles][4]    (block, adapter, lo, n): each run cut at block
 *                           boundaries, lo and n relative to the block;
 *                           unused (-1, -1, 0, 0)
 *   block_tile_start [nblk+1]  index of the first tile of block >= b
 *   counts [4]              num_padded, n_lora_seg, n_tiles, 0
 * with R = n_tokens * k, cap = BM * ceil((R + min(E, R) * (BM - 1)) / BM),
 * nblk = cap / BM, max_seg = min(R, E * NA), max_tiles = nblk + max_seg.
 * --------------------------------------------------------------------- */
typedef struct moelora_layout {
    int32_t block_m, cap, nblk, max_seg, max_tiles, reserved;
    size_t off_topk_ids, off_topk_w, off_sorted_rows, off_block_expert,
        off_seg_start, off_lora_seg, off_tiles, off_block_tile_start,
        off_counts, off_error;
} moelora_layout;

/* The layout a forward of n_tokens tokens uses (host only). */
MOELORA_API moelora_status moelora_workspace_layout(moelora_plan_t plan, int32_t n_tokens,
                                        moelora_layout *layout);

/* Synchronise `stream`, then copy the device error word of the last forward
 * that used `workspace` into *error_bits (MOELORA_DEVERR_* bits). */
MOELORA_API moelora_status moelora_read_device_error(moelora_plan_t plan,
                                         const void *workspace,
                                         int32_t *error_bits,
                                         moelora_stream_t stream);

/* A one-line description of the kernels and tiles a forward of n_tokens
 * tokens uses (for logs); NUL-terminated, truncated to buf_len. */
MOELORA_API moelora_status moelora_plan_info(moelora_plan_t plan, int32_t n_tokens,
                                 char *buf, size_t buf_len);

/* Stage timing.  Between moelora_timing_begin and moelora_timing_end the
 * plan records HIP events around each stage of every forward (at most
 * max_calls forwards), on the forward's stream.  moelora_timing_end
 * synchronises, writes the summed milliseconds of each stage into
 * stage_ms[0..n_stages) (stages: 0 routing + alignment, 1 gate_up shrink,
 * 2 gate_up GEMM + expand + SiLU*up, 3 down shrink, 4 down GEMM + expand,
 * 5 top-k combine) and the number of timed forwards into *n_calls.  Events
 * are created in begin and destroyed in end, so timed forwards still
 * allocate nothing.  A plan in timing mode must not be used from two
 * threads at once. */
#define MOELORA_N_STAGES 6
MOELORA_API moelora_status moelora_timing_begin(moelora_plan_t plan, int32_t max_calls);
MOELORA_API moelora_status moelora_timing_end(moelora_plan_t plan, double *stage_ms,
                                  int32_t n_stages, int32_t *n_calls);

#ifdef __cplusplus
}
#endif

#endif /* MOELORA_H */
