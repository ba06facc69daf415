/*
 * moelora.h -- C ABI of the routed MoE expert layer with rank-r side-LoRA
 * (forward and backward) on one AMD MI355X (gfx950).
 *
 * What the calls compute follows DeepGEMM PR #9 "feat(mega): add fused shared
 * side-LoRA kernels" (section "Historical implementation": Summary and
 * Correctness coverage) and PR #17 "Align MegaMoE training with upgraded
 * K-grouped TMA and layouts" (Summary):
 *   - routes are dispatched into an expert-contiguous pool, each expert padded
 *     to BLOCK_M rows, padding rows zeroed;
 *   - per route (t, j) with expert e and u = x_t:
 *       g = W1_e u + s B1_e (A1 u),  v = W3_e u + s B3_e (A3 u),
 *       h = silu(g) * v,             y = W2_e h + s B2 (A2_e h),
 *       out_t = sum_j w[t, j] y_(t, j)
 *     with A1, A3, B2 shared by all experts and B1, B3, A2 expert-local;
 *   - the backward returns grad-x and the router gradients in source-token
 *     order and the six adapter gradients (no frozen-weight gradients unless
 *     asked for), with padding rows kept out of every reduction;
 *   - unsupported modes and short workspaces are rejected before any launch.
 *
 * Conventions for every call:
 *   - All tensor pointers are DEVICE pointers, row-major, densely packed, and
 *     16-byte aligned.  bf16 is stored as uint16 bit patterns.
 *   - The caller owns every buffer.  The library never allocates, frees or
 *     keeps a pointer after a call returns.
 *   - Work is queued on `stream` (a hipStream_t; NULL = the null stream) and
 *     the call returns without waiting for the device.
 *   - Arguments are validated on the host first.  On any error nothing is
 *     written and no kernel is launched.
 *   - Outputs are overwritten, never accumulated; empty experts and dropped
 *     routes get exact zeros.
 *   - Calls that share a workspace or outputs must be ordered on one stream.
 *   - The forward and backward run independent parts of their work on a
 *     second stream of the device that the library creates on first use
 *     (non-blocking, default priority), ordered against the caller's stream
 *     by events: it waits for the caller's stream at the call's start, and
 *     the caller's stream waits for it before the call's last kernel, so in
 *     the caller's stream order the call's work is complete as before.
 *     Calls on one device hold a host lock while they enqueue.  While the
 *     caller's stream is being captured into a graph, and in
 *     moe_lora_forward_noalloc, every kernel runs on the caller's stream.
 */
#ifndef MOELORA_H
#define MOELORA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t moe_status;
#define MOE_OK 0
#define MOE_ERR_INVALID (-1)     /* bad shape, pointer, alignment or pool */
#define MOE_ERR_UNSUPPORTED (-2) /* a mode this build does not implement */
#define MOE_ERR_WORKSPACE (-3)   /* saved/scratch buffer smaller than required */
#define MOE_ERR_HIP (-4)         /* a HIP launch or attribute call failed */

#define MOE_ACT_SWIGLU 0         /* h = silu(g) * v, silu(g) = g sigmoid(g) */
#define MOE_ACT_GEGLU 1          /* h = gelu(g) * v, gelu(g) = g Phi(g) (exact GELU,
                                    Phi the standard normal distribution function);
                                    other values: UNSUPPORTED */
#define MOE_BASE_BF16 0          /* W13 / W2 in bf16 */
#define MOE_BASE_MXFP4 1         /* W13 / W2 as e2m1 with e8m0 scales per 32 along K */

/* Device status word of the saved workspace: the int32 at byte offset
 * MOE_SAVED_STATUS_OFFSET of `saved`, cleared by every moe_lora_forward and
 * raised by its kernels (read it after the forward, on the same stream).
 *   MOE_SAVED_FP16_RANGE  the gate/up pre-activations g, v are saved in fp16
 *     for the backward.  Without a clamp they must stay below 65504 in
 *     magnitude; the bit is set when some |g| or |v| reached 65520 or more
 *     (it rounds to infinity in fp16).  The forward's `out` is still right
 *     (the activation uses the fp32 values) but a backward from this saved
 *     state returns non-finite gradients.  With a clamp 0 < c < 65504 such
 *     values are clipped to c like any other value beyond it, and the bit is
 *     never set. */
#define MOE_SAVED_STATUS_OFFSET 0
#define MOE_SAVED_FP16_RANGE 1

/* Shape and options of one layer call.
 *   T tokens, H hidden, I intermediate, E local experts, topk routes per token,
 *   rank r of the side adapters, scale s of the adapter deltas (0 => plain MoE).
 *   block_m: pool padding granularity; 0 asks the library (see moe_lora_block_m),
 *     otherwise one of 16, 32, 64, 96, 128, 192, 240.
 *   activation: MOE_ACT_SWIGLU or MOE_ACT_GEGLU (the gated activations the
 *     pages list: PR #17 Summary; PR #9, "Correctness coverage").
 *   clamp: activation clamp c: when 0 < c < +inf both pre-activations are
     clipped to [-c, c] before the gated activation, h = f(clip(g)) clip(v),
     and the clip passes the gradient only where |x| <= c (the pages name the
     clamp -- PR #9 "Correctness coverage", production clamp = 10 -- without
     defining it; this is the plainest reading).  c <= 0 or +inf: no clamp;
     NaN: MOE_ERR_INVALID.  The clip decision is taken on the fp16-rounded
     pre-activation the forward saves, so forward and backward agree.
 * Supported: T >= 1, H % 256 == 0, I % 256 == 0, 1 <= E <= 512,
 *   1 <= topk <= 16, 1 <= rank <= 256 (a rank that is not a multiple of 8
 *   runs on copies of the factors widened with zero rows or columns to the
 *   next multiple, kept in the scratch workspace; the extra terms are exact
 *   zeros and the gradients are cut back to the caller's rank), T*H*2 and 4*I*H
 *   below 2^31 bytes (one 32-bit buffer offset per token-row tensor and per
 *   expert's weights).  Other values: MOE_ERR_UNSUPPORTED (non-positive sizes:
 *   MOE_ERR_INVALID).  base_format: MOE_BASE_BF16 or MOE_BASE_MXFP4. */
typedef struct moe_lora_desc {
  int32_t T, H, I, E, topk, rank;
  int32_t block_m;
  float scale;
  int32_t activation;
  float clamp;
  int32_t base_format;
} moe_lora_desc;

/* The dispatch pool written by build_pool (device int32 arrays).
 *   counts[E]          routes per expert
 *   offsets[E+1]       first pool row of each expert; offsets[E] = pool rows in use
 *   route_to_row[T*k]  pool row of route f = t*k + j, -1 if dropped
 *   row_to_route[capacity]  route of each pool row, -1 for padding and unused rows
 *   capacity           rows of row_to_route; must equal moe_lora_pool_capacity()
 *   block_m            the resolved BLOCK_M the pool was built with */
typedef struct moe_pool {
  const int32_t* counts;
  const int32_t* offsets;
  const int32_t* route_to_row;
  const int32_t* row_to_route;
  int64_t capacity;
  int32_t block_m;
} moe_pool;

/* Layer parameters (device, bf16 unless noted; nn.Linear [out, in] layout):
 *   W13 [E, 2I, H]  rows 0..I-1 = W1 (gate), rows I..2I-1 = W3 (up)
 *   W2  [E, H, I]
 *   A1, A3 [r, H]   shared;   B1, B3 [E, I, r] expert-local
 *   A2  [E, r, I]   expert-local;   B2 [H, r] shared
 *   W13_scale, W2_scale: e8m0 block scales for MOE_BASE_MXFP4, NULL for bf16.
 *   W13T, W2T, W13P, W2P: optional transformed copies of the frozen base,
 *     written once by moe_lora_transform_base and reused by every call
 *     (PR #9 Summary: reusable transformed weights), in a layout private to
 *     the library: the weight tiles of one GEMM pipeline stage stored as the
 *     bytes it loads, one stage after another, so that each stage reads one
 *     contiguous block (32 KB of bf16, or 9 KB of MXFP4 codes and scales)
 *     instead of a short run from each of 256 rows.
 *       W13T, W2T: W13[e]^T, W2[e]^T for the backward's two data-gradient
 *         GEMMs, E x 2I x H and E x H x I bf16 values (for an MXFP4 base, of
 *         the dequantised values); without them (NULL) the backward
 *         transposes W13 / W2 on the fly (an MXFP4 base also expanded to
 *         bf16).  The forward ignores them.
 *       W13P, W2P: W13, W2 for the forward's two base GEMMs: E x 2I x H and
 *         E x H x I bf16 values; for MOE_BASE_MXFP4, E*2I*H*9/16 and
 *         E*H*I*9/16 bytes (the e2m1 codes and e8m0 scales).  The backward
 *         ignores them.
 *     Results are bitwise the same with or without any of them; their
 *     contents must come from moe_lora_transform_base on the same W13 / W2.
 *     Each may be given alone; 16-byte aligned. */
typedef struct moe_lora_params {
  const void* W13;
  const void* W2;
  const uint8_t* W13_scale;
  const uint8_t* W2_scale;
  const void *A1, *A3, *B1, *B3, *A2, *B2;
  const void* W13T;
  const void* W2T;
  const void* W13P;
  const void* W2P;
} moe_lora_params;

/* Gradient outputs (device bf16, same layouts as the parameters).  The six
 * adapter gradients are required.  dW13 [E, 2I, H] and dW2 [E, H, I] are the
 * optional frozen-weight gradients of the ordinary path (PR #9, "Matched
 * old/new performance"): dW13_e = sum over e's routes of [dg; dv] x_t^T,
 * dW2_e = sum of (w go_t) h^T, contracted over the expert's rows in pool
 * order; an expert without routes gets exact zeros.  NULL skips each; a
 * non-NULL pointer must be 16-byte aligned (else MOE_ERR_INVALID).  With an
 * MXFP4 base they are the gradients with respect to the dequantised
 * weights. */
typedef struct moe_lora_grads {
  void *dA1, *dA3, *dB1, *dB3, *dA2, *dB2;
  void *dW13, *dW2;
} moe_lora_grads;

/* Human-readable name of a status code (static string). */
const char* moe_lora_status_string(moe_status status);

/* Library version, e.g. 100 for 0.1.0. */
int32_t moe_lora_version(void);

/* BLOCK_M used for `desc` (resolves block_m == 0 to the library's choice).
 * PR #17 Summary: the block size is queried from the library, not duplicated
 * by callers; forward and backward use the same pool. */
moe_status moe_lora_block_m(const moe_lora_desc* desc, int32_t* block_m);

/* Rows of row_to_route to allocate: T*k + min(E, T*k) * (BLOCK_M - 1), the
 * largest pool any routing can produce. */
moe_status moe_lora_pool_capacity(const moe_lora_desc* desc, int64_t* rows);

/* Bytes of the two workspaces:
 *   saved   -- written by moe_lora_forward, read by moe_lora_backward; holds
 *              the status word (MOE_SAVED_STATUS_OFFSET), a copy of the layer
 *              input (the saved-X reuse of PR #9, "2026-09-20" -> What
 *              changed), the gate/up pre-activations in fp16 (|g|, |v| must
 *              stay below 65504 without a clamp: MOE_SAVED_FP16_RANGE) and
 *              the activations.
 *   scratch -- temporary space of moe_lora_forward and moe_lora_backward
 *              (nothing in it survives a call; both need the full size). */
moe_status moe_lora_workspace_size(const moe_lora_desc* desc, size_t* saved_bytes,
                                   size_t* scratch_bytes);

/* Build the dispatch pool from top-k expert ids (PR #9, "2026-09-21: restore
 * wide-K wgrad safely" -> Implementation: true physical expert offsets, groups
 * never rounded into a neighbour; "Historical implementation" -> Summary:
 * padding zeroed).
 *   topk_idx [T, k] int32: expert id, or -1 for a dropped route.  Ids outside
 *     [-1, E) are dropped as well and counted into *device_error (device
 *     int32, may be NULL), which the call overwrites.
 *   Rows of one expert follow ascending route index t*k + j (deterministic).
 *   counts, offsets, route_to_row, row_to_route: outputs as in moe_pool. */
moe_status build_pool(const moe_lora_desc* desc, const int32_t* topk_idx, int32_t* counts,
                      int32_t* offsets, int32_t* route_to_row, int32_t* row_to_route,
                      int64_t capacity, int32_t* device_error, void* stream);

/* Write the transformed base weights of moe_lora_params from params->W13 /
 * params->W2 (the adapter factors are not read): W13T and W2T (E*2I*H and
 * E*H*I bf16 values: the transposed weights for the backward; for
 * MOE_BASE_MXFP4 the dequantised weights e2m1 x 2^(e-127), exact in bf16,
 * read from the packed W13 / W2 and their scales, both required) and W13P,
 * W2P (the forward's weights: the same sizes for a bf16 base; for
 * MOE_BASE_MXFP4 E*2I*H*9/16 and E*H*I*9/16 bytes of codes and scales).
 * Any output may be NULL (skipped); outputs are 16-byte aligned device
 * buffers that overlap no input and no other output.  Queued on `stream`
 * like every call. */
moe_status moe_lora_transform_base(const moe_lora_desc* desc, const moe_lora_params* params, void* W13T,
                                   void* W2T, void* W13P, void* W2P, void* stream);

/* Two-term FP6 (E2M3) split of bf16 rows, the activation operand of the
 * MXFP4 base's scaled fp6 x fp4 matrix products (PR #9 "Historical
 * implementation" -> Summary: native MXFP4 base with bf16 side adapters, the
 * activations keeping bf16 precision).  moe_lora_forward runs it internally
 * on x and on the activations h; this call exposes it alone.
 *   src [rows, K] bf16 (K % 64 == 0, else MOE_ERR_UNSUPPORTED).
 *   Per row and aligned 32-block: s1 = 2^E1 with E1 the smallest integer such
 *   that max|x| <= 7.5 s1 (E1 = -127 for an all-zero block), q1 = E2M3(x/s1)
 *   rounded to nearest, ties to even (OCP MX v1.0 FP6 E2M3: bias 1,
 *   subnormals m/8, largest 7.5; code 8e + m, sign in bit 5), r = x - s1 q1
 *   (exact), (s2, q2) from r the same way; |x - (s1 q1 + s2 q2)| <=
 *   2^-8 max(|x|, s1).
 *   codes [rows, 2K bytes]: per 64-element chunk c, 128 bytes; term t (q1,
 *     then q2) at 64t; the 32 six-bit codes of the chunk's 32-block h packed
 *     into six little-endian dwords (element i in bits 6i .. 6i+5), dwords
 *     0-3 at 64t + 16h and dwords 4-5 at 64t + 32 + 8h; bytes 64t + 48 ..
 *     64t + 63 are not written;
 *   scale_words [K/64, rows] uint32 (stage-major: the words of one chunk
 *     for all rows are consecutive): per chunk, bytes {E1+127 of its first
 *     32-block, of its second, E2+127 of the first, of the second}.
 *   src, codes 16-byte aligned, scale_words 4-byte aligned, no overlaps. */
moe_status moe_lora_split_e2m3x2(const void* src, int64_t rows, int32_t K, void* codes, void* scale_words,
                                 void* stream);

/* Forward of the layer.
 *   x [T, H] bf16, topk_w [T, k] fp32 router weights (used as given),
 *   out [T, H] bf16 (overwritten), saved / scratch per moe_lora_workspace_size
 *   (16-byte aligned; a short one returns MOE_ERR_WORKSPACE).
 *   `pool` must come from build_pool with the same desc and topk ids.
 *   x, out and the workspaces must not overlap. */
moe_status moe_lora_forward(const moe_lora_desc* desc, const moe_pool* pool, const void* x,
                            const float* topk_w, const moe_lora_params* params, void* out,
                            void* saved, size_t saved_bytes, void* scratch, size_t scratch_bytes,
                            void* stream);

/* moe_lora_forward without a scratch argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid allocation).  Same arguments, checks and results as
 * moe_lora_forward (bitwise); the forward's temporary tensors live instead in
 * a device array inside the library, 64 MiB on every device the library runs
 * on, held until the process ends.  The call allocates and frees nothing.
 *   - A layer whose forward needs more than 64 MiB of scratch returns
 *     MOE_ERR_WORKSPACE before any launch (the production share needs far
 *     more: use moe_lora_forward there; the token-sweep shapes up to a few
 *     hundred tokens fit).
 *   - All calls on one device share that device's array: calls that overlap
 *     on one device (different streams, concurrent threads) race.  Order them
 *     on one stream.
 *   - The first call on a device looks the array's address up (a HIP
 *     symbol query, no allocation); failure returns MOE_ERR_HIP. */
moe_status moe_lora_forward_noalloc(const moe_lora_desc* desc, const moe_pool* pool, const void* x,
                                    const float* topk_w, const moe_lora_params* params, void* out,
                                    void* saved, size_t saved_bytes, void* stream);

/* Backward of the layer for L = <grad_out, out>.
 *   grad_out [T, H] bf16; topk_w and params as given to the forward; `saved`
 *   as the forward left it (read only, may be reused by repeated calls).
 *   grad_x [T, H] bf16, grad_topk_w [T, k] fp32 (0 for dropped routes) and the
 *   gradients in `grads` are overwritten.  The result is a deterministic
 *   function of the inputs (bitwise repeatable). */
moe_status moe_lora_backward(const moe_lora_desc* desc, const moe_pool* pool,
                             const void* grad_out, const float* topk_w,
                             const moe_lora_params* params, const void* saved,
                             size_t saved_bytes, void* grad_x, float* grad_topk_w,
                             const moe_lora_grads* grads, void* scratch, size_t scratch_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * Several adapters in one pass (OpenPipe/ART PR #1139, Behavior: several
 * adapters share one MoE pass; the router runs once per adapter; the
 * dispatched expert rows carry adapter IDs so that each adapter's own LoRA
 * factors serve its rows; Validation: the fused pass equals running the
 * adapters one after another, bit for bit).
 *
 * The T tokens of a call form `count` roots, one per adapter: root a is the
 * tokens offsets[a] .. offsets[a+1]-1 (contiguous; an empty root is
 * allowed), and every route of a token carries its root's adapter.  For each
 * root the calls compute exactly what the single-adapter calls above compute
 * on that root's tokens with adapter a's factors: outputs, grad-x and router
 * gradients by token, and each adapter's factor gradients over its own root
 * (an adapter with an empty root gets exact zeros).  The base W13 / W2 (and
 * W13T / W2T, the MXFP4 scales, s and every desc field) are common.
 *
 * Parameters and gradients are the single-adapter tensors stacked over the
 * adapters: A1, A3 [count, r, H]; B1, B3 [count, E, I, r]; A2 [count, E, r,
 * I]; B2 [count, H, r]; likewise dA1 .. dB2.  The frozen-weight gradients
 * dW13 / dW2 are not offered with count > 1 (MOE_ERR_UNSUPPORTED).
 *
 * The pool groups rows by (expert e, adapter a) as group g = e * count + a:
 * counts / offsets have E * count (+1) entries, and the capacity is
 * T*k + min(E * count, T*k) * (BLOCK_M - 1) (moe_lora_multi_pool_capacity).
 * A pool built by build_pool_multi serves only the *_multi calls with the
 * same adapters.  count = 1 with offsets {0, T} is exactly the single-adapter
 * path.
 * ------------------------------------------------------------------------ */
#define MOE_MAX_ADAPTERS 64

/* offsets: HOST int32 array of count + 1 entries, 0 = offsets[0] <= ... <=
 * offsets[count] = T (else MOE_ERR_INVALID); 1 <= count <= MOE_MAX_ADAPTERS
 * (more: MOE_ERR_UNSUPPORTED).  Read during the call only. */
typedef struct moe_adapters {
  int32_t count;
  const int32_t* offsets;
} moe_adapters;

moe_status moe_lora_multi_pool_capacity(const moe_lora_desc* desc, const moe_adapters* adapters,
                                        int64_t* rows);
moe_status moe_lora_multi_workspace_size(const moe_lora_desc* desc, const moe_adapters* adapters,
                                         size_t* saved_bytes, size_t* scratch_bytes);
/* build_pool with (expert, adapter) groups: counts [E*count], offsets
 * [E*count + 1]; rows of a group follow ascending route index. */
moe_status build_pool_multi(const moe_lora_desc* desc, const moe_adapters* adapters, const int32_t* topk_idx,
                            int32_t* counts, int32_t* offsets, int32_t* route_to_row, int32_t* row_to_route,
                            int64_t capacity, int32_t* device_error, void* stream);
/* moe_lora_forward / moe_lora_backward over the roots (adapters != NULL). */
moe_status moe_lora_forward_multi(const moe_lora_desc* desc, const moe_adapters* adapters, const moe_pool* pool,
                                  const void* x, const float* topk_w, const moe_lora_params* params, void* out,
                                  void* saved, size_t saved_bytes, void* scratch, size_t scratch_bytes,
                                  void* stream);
moe_status moe_lora_backward_multi(const moe_lora_desc* desc, const moe_adapters* adapters, const moe_pool* pool,
                                   const void* grad_out, const float* topk_w, const moe_lora_params* params,
                                   const void* saved, size_t saved_bytes, void* grad_x, float* grad_topk_w,
                                   const moe_lora_grads* grads, void* scratch, size_t scratch_bytes,
                                   void* stream);

/* ------------------------------------------------------------------------
 * The router: what a layer call takes as topk_idx and topk_w, the load of
 * each expert and its balance loss, and the gradient of all of them.
 *
 * Token t of root a (roots as in moe_adapters; NULL adapters: one root) with
 * logits l_te over E experts is ACTIVE when valid[t] != 0, no logit of it is
 * NaN or +inf, and at least one is above -inf.  For an active token
 *   idx_t   = the topk largest logits, descending, equals in ascending expert
 *             order; an expert at -inf is never taken (missing routes: -1),
 *   p_te    = exp(l_te) / sum_e' exp(l_te')          (max-shifted, fp32),
 *   w_tj    = p at idx_tj, divided by their sum if `renorm`; 0 where idx is -1.
 * An inactive token gets idx -1, w 0 and takes part in nothing below.
 *   counts[a, e] = routes of root a's tokens to e,   n_a = active tokens of a,
 *   loss[a]  = E / (topk n_a^2) sum_e counts[a, e] sum_t p_te    (n_a = 0: 0),
 * the product of each expert's share of the routes and its mean probability
 * (1 at perfect balance with topk routes per token).  With several roots the
 * router runs once per root (OpenPipe/ART PR #1139, Behavior).
 *
 * Backward, for dL/dw = grad_w and dL/dloss = grad_loss (either may be NULL:
 * zero), the counts taken as constants:
 *   u_te = grad_loss[a] E / (topk n_a^2) counts[a, e]
 *   dl_te = p_te (u_te - sum_e' p u) + the top-k term:
 *     renorm:  at e = idx_tj: w_tj (grad_w_tj - sum_i w_ti grad_w_ti)
 *     else:    p_te (G_te - sum_e' p G), G = grad_w at the chosen experts.
 * grad_logits has the logits' type and is 0 for inactive tokens.
 *
 * Supported: 1 <= T <= 2^30, 1 <= E <= 512, 1 <= topk <= min(16, E),
 * T * E < 2^31, T * topk < 2^31 (others: MOE_ERR_UNSUPPORTED; topk > E or non-positive
 * sizes: MOE_ERR_INVALID).  Sums over tokens run in a fixed order: results
 * are bitwise repeatable.
 * ------------------------------------------------------------------------ */
#define MOE_TYPE_F32 0
#define MOE_TYPE_BF16 1

typedef struct moe_router_desc {
  int32_t T, E, topk;
  int32_t logits_type; /* MOE_TYPE_F32 or MOE_TYPE_BF16 */
  int32_t renorm;      /* 0 or 1 */
} moe_router_desc;

/* Bytes of the workspace of moe_router_forward (nothing in it survives the
 * call).  adapters may be NULL (one root). */
moe_status moe_router_workspace_size(const moe_router_desc* desc, const moe_adapters* adapters, size_t* bytes);

/* logits [T, E]; valid [T] uint8 or NULL (every token valid); outputs
 * topk_idx [T, topk] int32, topk_w [T, topk] fp32, counts [roots, E] int32,
 * active [roots] int32 (n_a), loss [roots] fp32; device_error (device int32,
 * may be NULL) is overwritten with the number of valid tokens dropped for a
 * NaN or +inf logit.  logits and workspace 16-byte aligned, the others by
 * their element. */
moe_status moe_router_forward(const moe_router_desc* desc, const moe_adapters* adapters, const void* logits,
                              const uint8_t* valid, int32_t* topk_idx, float* topk_w, int32_t* counts,
                              int32_t* active, float* loss, int32_t* device_error, void* workspace,
                              size_t workspace_bytes, void* stream);

/* topk_idx, counts and active as moe_router_forward wrote them for the same
 * logits and valid; grad_topk_w [T, topk] fp32 or NULL (not used where the id is -1), grad_loss [roots]
 * fp32 or NULL; grad_logits [T, E] of the logits' type (overwritten; may be
 * the logits' own buffer). */
moe_status moe_router_backward(const moe_router_desc* desc, const moe_adapters* adapters, const void* logits,
                               const uint8_t* valid, const int32_t* topk_idx, const int32_t* counts,
                               const int32_t* active, const float* grad_topk_w, const float* grad_loss,
                               void* grad_logits, void* stream);

/* ------------------------------------------------------------------------
 * One AdamW step over many tensors (the six adapter factors of one or more
 * layers and adapters).  Per element, with g = grad_scale * grad:
 *   m <- beta1 m + (1 - beta1) g        v <- beta2 v + (1 - beta2) g^2
 *   p <- p (1 - lr weight_decay) - lr (m / bias1) / (sqrt(v / bias2) + eps)
 * with bias1 = 1 - beta1^step, bias2 = 1 - beta2^step, in fp32; p's whole
 * change, decay included, is formed first and subtracted once.  p is the
 * fp32 master copy if there is one (then `param` receives its rounding), else
 * `param` itself.
 *
 * state_bits 32: m, v fp32.  state_bits 8: per run of 128 elements of a
 * tensor (the last one may be short) m is e4m3 codes times one fp32 scale
 * (max|m| / 448) and v is e5m2 codes times one fp32 scale (max v / 57344);
 * the step itself uses the unrounded m and v.  Codes are rounded at random:
 * y = x * (top * (1 / max)), top = 448 or 57344 (each operation rounded to
 * fp32, as in the moments above), is clamped to [-top, top] and becomes
 * floor(|y| / s + u) * s with y's sign: s is the format's step at y (e4m3 2^-9
 * below 2^-6, e5m2 2^-16 below 2^-14), u one of 2^16 equally likely multiples
 * of 2^-16 in [0, 1).  On the mean a code is y, also below the normal range,
 * to 2^-16 s.  Without it a decaying average would stop moving once a step
 * changes it by less than half a code.  One exception: a positive v below
 * 2^-16 / 57344 (2.7e-10) of its run's largest is held as that, the lowest
 * code (its element moves less than with fp32 moments), so that in a run that
 * does not count as zero (see below) no m is divided by eps alone.  The random
 * bits of element i of a tensor are a fixed mix of i and `seed`; pass another
 * seed each step.
 *   x0 = i * 0x9E3779B9 + seed, x1 = (x0 ^ x0 >> 16) * 0x6A09E667,
 *   x2 = (x1 ^ x1 >> 15) * 0xBB67AE85, r = x2 ^ x2 >> 16 (mod 2^32):
 *   u = bits 0-15 / 2^16 for m, bits 16-31 / 2^16 for v.
 * A run whose new moments are not finite gets a non-finite scale; one whose
 * largest moment is below 2^-100 counts as zero.
 * All-zero codes and scales are the state before the first step.
 * ------------------------------------------------------------------------ */
typedef struct moe_adamw_tensor {
  void* param;       /* [n] of param_type, updated */
  float* master;     /* [n] fp32 or NULL (bf16 parameters only; all tensors of a call alike) */
  const void* grad;  /* [n] of grad_type */
  void* m;           /* [n] fp32, or e4m3 codes */
  void* v;           /* [n] fp32, or e5m2 codes */
  float* m_scale;    /* [ceil(n / 128)] with state_bits 8, else NULL */
  float* v_scale;
  int64_t n;         /* 0 to 2^34 (more: MOE_ERR_UNSUPPORTED); 0: skipped, pointers not looked at */
} moe_adamw_tensor;

/* What changes from step to step, in device memory: for steps captured into
 * a graph and replayed with other values. */
typedef struct moe_adamw_control {
  float lr, bias1, bias2, grad_scale;
  uint32_t seed;
} moe_adamw_control;

typedef struct moe_adamw_desc {
  int32_t param_type, grad_type; /* MOE_TYPE_* */
  int32_t state_bits;            /* 32 or 8 */
  uint32_t seed;                 /* read with state_bits 8 */
  double lr, beta1, beta2, eps, weight_decay, grad_scale;
  int64_t step;                  /* 1 for the first step */
  const moe_adamw_control* control; /* DEVICE pointer or NULL: replaces lr, step's biases, grad_scale and seed */
} moe_adamw_desc;

/* Update `count` tensors (HOST array, read during the call).  Pointers of
 * non-empty tensors 16-byte aligned (scales 4-byte); no buffer of the call
 * may overlap another one that it writes (within a tensor this is checked).
 * lr, weight_decay >= 0, eps > 0,
 * betas in [0, 1), step >= 1, all finite in fp32, else MOE_ERR_INVALID. */
moe_status moe_adamw_step(const moe_adamw_desc* desc, const moe_adamw_tensor* tensors, int32_t count, void* stream);

/* ------------------------------------------------------------------------
 * Expert products in 8-bit floating point with one fp32 scale for each block
 * of 128: the base of a layer stored as e4m3 codes with a scale per 128 x 128
 * block of a weight, activations as e4m3 codes with a scale per row and 128
 * columns.  For pool row r of expert e (rows as build_pool laid them out)
 *   out[r, n] = sum_c sa[a(r), c] sw[e, n / 128, c] sum_{k in block c} a[a(r), k] w[e, n, k]
 * in fp32 over the blocks, rounded once to bf16.  Inside a block the matrix
 * core adds: it aligns 8 consecutive products a w to the largest exponent sum
 * among them and drops what lies below 2^-13 of it, and joins the groups of 8
 * in 24 bits (measured; far below the 2^-4 of the codes themselves).  The
 * order of all sums is fixed.  a(r) is the token
 * row_to_route[r] / topk (gate / up: tokens are gathered) or r itself (down,
 * and the gradients of pool rows).  The data gradient is the same product
 * with the transposed weight and its transposed scales.
 * E4M3 is OCP FP8 E4M3 (largest value 448, NaN 0x7F, no infinities).
 * ------------------------------------------------------------------------ */
#define MOE_FP8_PLAIN (-1)

/* Rows to codes and scales: per row and 128 columns scale = max|x| / 448 and
 * code = e4m3(x * (448 / max|x|)), to nearest, ties to even (fp32 arithmetic;
 * an all-zero block, or one with a maximum below 2^-100: scale 0, codes 0).
 * A block with a NaN or an infinity gets a non-finite scale.
 *   act MOE_FP8_PLAIN: src [rows, K] bf16, x = src;
 *   act MOE_ACT_SWIGLU / MOE_ACT_GEGLU: src [rows, 2K] bf16 = [gate | up],
 *     x = act(gate) * up in fp32.
 *   codes [rows, K] bytes, scales [rows, K / 128] fp32.  K % 128 == 0 (else
 *   MOE_ERR_UNSUPPORTED), K at most 65536, rows * K at most 2^35 - 2048, rows >= 0 (0: nothing is done). */
moe_status moe_fp8_quantize_rows(const void* src, int64_t rows, int32_t K, int32_t act, void* codes, float* scales,
                                 void* stream);

/* Weights W [E, N, K] bf16 to codes [E, N, K] and scales [E, N/128, K/128] by
 * 128 x 128 blocks (the same rounding), and, if both are given, the same
 * codes transposed per expert, codes_t [E, K, N] and scales_t [E, K/128,
 * N/128].  N, K % 128 == 0 and at most 65536, 1 <= E <= 512, N * K < 2^31. */
moe_status moe_fp8_quantize_weight(const void* W, int32_t E, int32_t N, int32_t K, void* codes, float* scales,
                                   void* codes_t, float* scales_t, void* stream);

typedef struct moe_fp8_desc {
  int32_t E, N, K; /* N, K % 128 == 0, at most 65536; 1 <= E <= 512; N * K < 2^31 */
  int32_t topk;    /* > 0: gather, row r reads activation row row_to_route[r] / topk; 0: row r */
  int64_t a_rows;  /* rows of a, at least 1: tokens (gather; a_rows * K < 2^31), at least the pool's rows in use otherwise */
} moe_fp8_desc;

/* out [pool->capacity, N] bf16: the rows of routes are written, padding and
 * unused rows are left as they were.  pool: counts, offsets and row_to_route
 * as build_pool wrote them (route_to_row is not read and may be NULL), E
 * experts, capacity = its allocated rows, 1 to 2^31 - 256.  a [a_rows, K], a_scales [a_rows,
 * K/128], w [E, N, K], w_scales [E, N/128, K/128].  A route whose activation
 * row is not below a_rows reads zeros; rows past the capacity are not
 * touched whatever the pool says.  Which kernel runs follows from the shapes;
 * a row's result does not depend on it (bitwise), nor on the other rows. */
moe_status moe_fp8_product(const moe_fp8_desc* desc, const moe_pool* pool, const void* a, const float* a_scales,
                           const void* w, const float* w_scales, void* out, void* stream);

/* ------------------------------------------------------------------------
 * Expert products in bf16 on the pool's rows, for weights outside a fused layer
 * call (a base trained with its own gradients, an unfused layer).  For pool row
 * r of expert e (rows as build_pool laid them out), with a(r) the token
 * row_to_route[r] / topk (topk > 0: tokens are gathered) or r itself (topk 0),
 *   out[r, n]  = sum_k a[a(r), k] w[e, n, k]      w [E, N, K]
 *                         (transposed: w[e, k, n], w [E, K, N])
 *   dw[e, n, k] = sum_{r of e} grad[r, n] a[a(r), k]   (+ dw, if `accumulate`)
 * in fp32, rounded once.  The data gradient of a product with weight [E, N, K]
 * is the transposed product of the same weight (with the two widths' names
 * exchanged): no second copy of the weight is needed.  The order of all sums
 * is fixed: results are bitwise repeatable, and a row of `out` does not depend
 * on the other rows' values.
 * ------------------------------------------------------------------------ */
typedef struct moe_expert_desc {
  int32_t E, N, K;    /* N, K % 8 == 0, at most 65536; 1 <= E <= 512; N * K < 2^30 */
  int32_t topk;       /* > 0: gather, row r reads activation row row_to_route[r] / topk; 0: row r */
  int64_t a_rows;     /* rows of a, at least 1; gather: a_rows * K < 2^30 */
  int32_t transposed; /* moe_expert_product: 1: w is [E, K, N] */
  int32_t out_type;   /* moe_expert_weight_grad: MOE_TYPE_* of dw */
  int32_t accumulate; /* moe_expert_weight_grad: 1: added to dw; 0: dw is overwritten, zeros for an expert without rows */
} moe_expert_desc;

/* out [pool->capacity, N] bf16: the rows of routes are written, padding and
 * unused rows are left as they were.  a [a_rows, K] bf16, w bf16.  pool:
 * counts, offsets and row_to_route as build_pool wrote them (route_to_row is
 * not read and may be NULL), capacity 1 to 2^31 - 256.  A route whose
 * activation row is not below a_rows reads zeros; rows past the capacity are
 * not touched whatever the pool says.  (capacity / 16 + E) * ceil(N / 16) <
 * 2^31. */
moe_status moe_expert_product(const moe_expert_desc* desc, const moe_pool* pool, const void* a, const void* w,
                              void* out, void* stream);

/* grad [pool->capacity, N] bf16 (rows of no route are not used), a [a_rows, K]
 * bf16, dw [E, N, K] of out_type; pool as in moe_expert_product. */
moe_status moe_expert_weight_grad(const moe_expert_desc* desc, const moe_pool* pool, const void* grad, const void* a,
                                  void* dw, void* stream);

/* ------------------------------------------------------------------------
 * The same in microscaled 4-bit floating point (OCP MX v1.0, MXFP4; the layout
 * of MOE_BASE_MXFP4): e2m1 codes, element 2i in the low nibble of byte i, and
 * one e8m0 exponent per 32 elements along the contraction axis.
 *
 * A block of 32 with largest magnitude m gets the exponent floor(log2 m) - 2
 * (held plus 127; a block of zeros, and one below 2^-125, holds 0) and each
 * element the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 times 2^exponent, ties to
 * the even code, what is beyond 6 to 6; a negative value that rounds to zero
 * is +0.  A block with a NaN or an infinity holds the exponent 255 (NaN).
 * ------------------------------------------------------------------------ */
/* act as in moe_fp8_quantize_rows: src [rows, K] bf16 (MOE_FP8_PLAIN) or
 * [rows, 2K] = [gate | up].  codes [rows, K / 2] bytes, exponents [rows, K / 32]
 * bytes.  K % 128 == 0 and at most 65536, 0 <= rows < 2^31 (0: nothing is
 * done), rows * K at most 2^35 - 2048. */
moe_status moe_mxfp4_quantize_rows(const void* src, int64_t rows, int32_t K, int32_t act, void* codes,
                                   void* exponents, void* stream);

/* W bf16 [E, N, K] to codes [E, N, K / 2] and exponents [E, N, K / 32] (blocks
 * along K) and, if both are given, of the transposed weight: codes_t [E, K,
 * N / 2] and exponents_t [E, K, N / 32] (blocks along N: other roundings of the
 * same weight), the data gradient's operand.  N, K % 128 == 0 and at most
 * 65536, 1 <= E <= 512, N * K < 2^31, E * N * K at most 2^35 - 2048. */
moe_status moe_mxfp4_quantize_weight(const void* W, int32_t E, int32_t N, int32_t K, void* codes, void* exponents,
                                     void* codes_t, void* exponents_t, void* stream);

/* What codes and exponents stand for, exactly, as bf16 [rows, K] (values below
 * bf16's smallest normal 2^-126 included; beyond its largest: infinities; 255:
 * NaN).  rows and K as in moe_mxfp4_quantize_rows. */
moe_status moe_mxfp4_dequantize(const void* codes, const void* exponents, int64_t rows, int32_t K, void* out,
                                void* stream);

typedef struct moe_mxfp4_desc {
  int32_t E, N, K; /* N % 32 == 0, K % 128 == 0, at most 65536; 1 <= E <= 512; N * K < 2^31 */
  int32_t topk;    /* as in moe_expert_desc */
  int64_t a_rows;  /* rows of a, at least 1; gather: a_rows * K < 2^32 */
} moe_mxfp4_desc;

/* out [pool->capacity, N] bf16 as moe_expert_product writes it, of a [a_rows,
 * K / 2], a_exponents [a_rows, K / 32], w [E, N, K / 2], w_exponents [E, N,
 * K / 32] (an MXFP4 base's W13 or W2 as the layer takes it): the products of
 * what the codes stand for, added by the scaled matrix instructions in fp32,
 * 128 at a time.  A NaN exponent makes its row's results NaN (a weight's: its
 * column's).  pool as in moe_expert_product; (capacity / 16 + E) * (N / 16) <
 * 2^31. */
moe_status moe_mxfp4_product(const moe_mxfp4_desc* desc, const moe_pool* pool, const void* a, const void* a_exponents,
                             const void* w, const void* w_exponents, void* out, void* stream);

/* ------------------------------------------------------------------------
 * One optimiser step with an orthogonalised update (momentum, then rounds of a
 * quintic polynomial that drive the update's singular values towards one) over
 * many matrices: adapter factors, each tensor [batch, m, n] a stack of matrices
 * (an expert-local factor: one matrix per expert).  Per matrix, with
 * g = grad_scale * grad:
 *   M <- momentum M + g,   U = g + momentum M (nesterov) or M,
 *   X <- U / (|U| + eps)            (|U| the root of the sum of its squares),
 *   `rounds` times  X <- a X + (b S + c S^2) X,  S = X X^T  (X^T X if m > n),
 *   p <- p - lr (rms sqrt(max(m, n)) X + weight_decay p).
 * M and p in fp32; p is the fp32 master copy if there is one (then `param`
 * receives its rounding), else `param` itself; p's whole change is formed first
 * and subtracted once.  X after the rounds is a polynomial of S times U: S and
 * the polynomial are formed in fp64, and multiply U in fp32 once.  A matrix of
 * zeros moves by its weight decay alone; one with a NaN or an infinity in U
 * becomes NaN and leaves the others alone.  All sums run in a fixed order:
 * results are bitwise repeatable.
 *
 * min(m, n) <= 256, m * n < 2^31, batch <= 2^18, batch * m * n < 2^40 (more:
 * MOE_ERR_UNSUPPORTED).
 * ------------------------------------------------------------------------ */
typedef struct moe_muon_tensor {
  void* param;       /* [batch, m, n] of param_type, updated */
  float* master;     /* fp32 or NULL (bf16 parameters only; all tensors of a call alike) */
  const void* grad;  /* of grad_type */
  float* momentum;   /* fp32, updated; zeros before the first step */
  int64_t batch;     /* 0: skipped, pointers not looked at */
  int32_t m, n;
} moe_muon_tensor;

/* What changes from step to step, in device memory: for steps captured into a
 * graph and replayed with other values. */
typedef struct moe_muon_control {
  float lr, grad_scale;
} moe_muon_control;

typedef struct moe_muon_desc {
  int32_t param_type, grad_type; /* MOE_TYPE_* */
  int32_t nesterov;              /* 0 or 1 */
  int32_t rounds;                /* 1 to 16 */
  double lr, momentum, weight_decay, rms, eps, grad_scale;
  double a, b, c;                /* the quintic's coefficients */
  const moe_muon_control* control; /* DEVICE pointer or NULL: replaces lr and grad_scale */
} moe_muon_desc;

/* Bytes of the workspace of moe_muon_step on the current device for these
 * tensors (nothing in it survives the call; pointers are not looked at). */
moe_status moe_muon_workspace_size(const moe_muon_desc* desc, const moe_muon_tensor* tensors, int32_t count,
                                   size_t* bytes);

/* Update `count` tensors (HOST array, read during the call).  Pointers of
 * non-empty tensors and the workspace 16-byte aligned; no buffer of the call
 * may overlap another one that it writes (within a tensor this is checked).
 * lr, weight_decay, rms >= 0, momentum in [0, 1), eps > 0, all finite in fp32,
 * else MOE_ERR_INVALID. */
moe_status moe_muon_step(const moe_muon_desc* desc, const moe_muon_tensor* tensors, int32_t count, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Optional per-kernel timing (the pages' backward carries an optional kernel
 * trace: PR #9 review-bot Overview).  When enabled, every kernel the library
 * launches is bracketed by two HIP events recorded on its launch stream; the
 * events are created on first use and reused.  Off by default.
 *   moe_lora_trace_enable(1 / 0)  turn recording on / off (process-wide)
 *   moe_lora_trace_collect()      wait for the recorded events and add their
 *                                 elapsed times to per-kernel totals
 *   moe_lora_trace_count()        number of kernels with totals
 *   moe_lora_trace_entry(i, ...)  name (static storage until the next reset),
 *                                 launch count and total milliseconds of entry i
 *   moe_lora_trace_reset()        clear the totals */
void moe_lora_trace_enable(int32_t on);
moe_status moe_lora_trace_collect(void);
int32_t moe_lora_trace_count(void);
moe_status moe_lora_trace_entry(int32_t i, const char** name, int64_t* launches, double* total_ms);
void moe_lora_trace_reset(void);

#ifdef __cplusplus
}
#endif

#endif /* MOELORA_H */
