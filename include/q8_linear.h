/*
 * q8_linear.h -- C ABI of the MI355X (gfx950) Q8_0 block-quantized weight linear.
 *
 * What is computed (sources are the pages describing the fucina engine):
 *   - "14. Model families and example applications", section 14.1 (Conventions shared
 *     by every family): LinearWeight keeps the GGUF dtype resident and the quant forms,
 *     Q8_0 among them, run packed kernels with no global dequantization at load; q/k/v
 *     are fused into one QKV matrix and gate/up into one gate_up matrix, one wider
 *     product per block.
 *   - Same page, section 14.2 (Qwen3 - dense and MoE): SwiGLU FFN; lockstep batch
 *     decode runs the trunk as one m = n pass that reads the weights once for all
 *     streams; the MoE FFN routes with softmax top-k (routerTopK, normalize_selected =
 *     norm_topk_prob) and runs the router-weighted SwiGLU mixture (moeSwiGluFfnSeq),
 *     grouped per expert, so that one pass over an expert's weights serves its tokens.
 *   - Same page, section 14.4 (Gemma 4 - text + MoE, "MoE expert kernels"): a
 *     counting-sort route plan and a per-token summation order kept fixed.
 *
 * Q8_0 tensor layout (the GGUF Q8_0 block; the pages name the format without spelling
 * it out): a row of length K is K/32 blocks of 34 bytes, each a little-endian IEEE
 * binary16 scale d followed by 32 signed 8-bit quants q; the weight is w = d * q.
 * Rows are contiguous: row n starts at byte n * (K/32) * 34.  Expert stacks are E such
 * matrices back to back.
 *
 * Conventions for every call below:
 *   - All tensor pointers are DEVICE pointers owned by the caller; nothing is freed,
 *     retained or allocated by the library.  Weights and inputs are only read.
 *   - Row-major float32 activations x [M][ldx] (the first K of each row used) and
 *     outputs [M][ld*].  Outputs are fully overwritten, never accumulated into.
 *   - stream is a hipStream_t passed as void* (NULL = the null stream).  Calls are
 *     asynchronous: they enqueue kernels and return; they never synchronize.
 *   - Arguments are validated on the host before anything is enqueued; on a bad
 *     argument the call returns an error code and enqueues nothing.  A launch failure
 *     reported by the HIP runtime returns Q8_ERR_DEVICE.  q8_last_error() then holds a
 *     thread-local description.
 *   - M = 0 (no rows) and N = 0 (no outputs) are valid and enqueue nothing.
 *   - K (and the MoE H and F) must be positive multiples of 256 (rows then stay 16-byte
 *     aligned: 8 blocks are 272 bytes); otherwise Q8_ERR_SHAPE.
 *   - Alignment: weight and x base pointers 16-byte aligned and ldx a multiple of 4;
 *     output pointers 4-byte aligned; otherwise Q8_ERR_ALIGN.
 *   - Results are deterministic: the same inputs give bit-identical outputs on every
 *     call (fixed summation orders, no floating-point atomics).
 *   - Calls are thread-safe; the only global state is the thread-local error text and
 *     a per-device cache of launch sizes.
 */
#ifndef Q8_LINEAR_H
#define Q8_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Raised where an existing call changes; calls that are only added leave it (a library
 * without one lacks its symbol). */
#define Q8_ABI_VERSION 8

typedef enum q8_status {
    Q8_OK = 0,
    Q8_ERR_NULL = 1,      /* a required pointer is NULL                                   */
    Q8_ERR_SHAPE = 2,     /* a size is negative, too large, or breaks the block structure */
    Q8_ERR_ALIGN = 3,     /* a pointer or leading dimension is misaligned                 */
    Q8_ERR_WORKSPACE = 4, /* workspace missing or smaller than q8_moe_workspace_bytes()   */
    Q8_ERR_DEVICE = 5     /* the HIP runtime reported an error                            */
} q8_status;

/* Version of this ABI (Q8_ABI_VERSION of the built library). */
int32_t q8_abi_version(void);

/* Static text for a status code. */
const char* q8_status_string(q8_status status);

/* Thread-local description of the last failure on this thread ("" if none). */
const char* q8_last_error(void);

/*
 * y = x . W^T  -- the packed-weight linear (section 14.1, LinearWeight; the fused QKV
 * and down projections use it directly).
 *   w_q8 : Q8_0 [n][k]          x : float32 [m][ldx]          y : float32 [m][ldy]
 *   n >= 0 outputs, k > 0 a multiple of 256, m >= 0 rows, ldx >= k, ldy >= n.
 * Arithmetic by batch size (the m-dependent kernel classes of section 14.2):
 *   m == 1      float32: per block t = sum q*x, acc = fma(d, t, acc), fixed butterfly;
 *   2..255      float32 in 16-row launches, per block t = sum q*x (the quants exact,
 *               one rounding per fma; the fp32 matrix cores' 4x4x1 form rounds like an
 *               fma), acc = fma(d, t, acc), in an order that depends only on k and n:
 *               k <= 4096 streams the weights once per launch on the matrix cores when
 *               its LDS fits (at k = 4096 on 256 CUs: n <= 129,024, fused f <= 47,104),
 *               a fixed sum over 16 pairs, then the 16-pair chunks in order; other calls
 *               run the float32 rows kernel (9..16 rows on its matrix-core form, the same
 *               bits); every row is bit-identical whatever the other rows are (for any m
 *               in 2..255), and agrees with the m == 1 result to reassociation;
 *   m >= 256    bf16 matrix cores (dense prefill): weights d*q and activations rounded
 *               to bf16 (nearest even), float32 accumulation and output.
 */
q8_status q8_linear(const void* w_q8, int64_t n, int64_t k,
                    const float* x, int64_t m, int64_t ldx,
                    float* y, int64_t ldy, void* stream);

/*
 * h = SiLU(x . W_gate^T) * (x . W_up^T) from one fused gate_up matrix (section 14.1 fuses
 * gate and up; section 14.2 gives the SwiGLU FFN).  SiLU(g) = g / (1 + exp(-g)).
 *   w_gate_up_q8 : Q8_0 [2f][k], gate rows [0, f) then up rows [f, 2f)
 *   x : float32 [m][ldx]          h : float32 [m][ldh], ldh >= f
 * Same rules (and the same arithmetic by batch size) as q8_linear otherwise.
 */
q8_status q8_linear_fused_gate_up_silu(const void* w_gate_up_q8, int64_t f, int64_t k,
                                       const float* x, int64_t m, int64_t ldx,
                                       float* h, int64_t ldh, void* stream);

/*
 * GGUF Q4_0 weights (the DGX Spark README, Features and Models: Q4_0 is read directly by
 * the quantized GEMV; section 14.1: the other ggml quant forms run their own packed
 * kernels).  The layout is the ggml one (the pages name the format only): per block of
 * 32 weights a little-endian binary16 scale d, then 16 bytes; weight j < 16 is the low
 * nibble of byte j, weight j + 16 the high nibble; w = d * (nibble - 8).  18 bytes per
 * block, rows of k/32 blocks back to back.
 *   q4_0_linear                     : y[m][n] = x . W^T,  W = Q4_0 [n][k]
 *   q4_0_linear_fused_gate_up_silu  : h = SiLU(x . W_gate^T) * (x . W_up^T), W = Q4_0 [2f][k]
 * Arguments, rules and errors as for q8_linear / q8_linear_fused_gate_up_silu.  Two or
 * more rows run the float32 rows kernel in 8-row launches (weights w = d*(q-8) exact in
 * float32, one fma per weight and row, the per-output order depends only on k: those rows
 * are bit-identical whatever m is).  One row with k <= 4096 on a matrix with at least 16
 * row groups per CU runs the one-row kernel (per block t = sum nibble*x, then
 * acc += d*(t - 8*sum x)), whose rows agree with the multi-row results to float32
 * reassociation; other one-row calls run the rows kernel.
 */
q8_status q4_0_linear(const void* w_q4_0, int64_t n, int64_t k,
                      const float* x, int64_t m, int64_t ldx,
                      float* y, int64_t ldy, void* stream);
q8_status q4_0_linear_fused_gate_up_silu(const void* w_gate_up_q4_0, int64_t f, int64_t k,
                                         const float* x, int64_t m, int64_t ldx,
                                         float* h, int64_t ldh, void* stream);

/*
 * GGUF k-quant weights, Q4_K, Q5_K and Q6_K ("14. Model families and example
 * applications", section 14.1: Q4_K, Q5_K and Q6_K run their own packed kernels; the DGX
 * Spark README, Features: the engine reads Q4_K and Q6_K blocks directly in its quantized
 * GEMV, without dequantizing the model at load).  The pages name the formats only; the
 * layouts are the ggml ones, super-blocks of 256 weights along k, rows of k/256
 * super-blocks back to back:
 *   Q4_K, 144 bytes: binary16 d, binary16 dmin, 12 bytes holding eight 6-bit (scale, min)
 *     pairs (sub-block j < 4: bits 0..5 of bytes j and j+4; j >= 4: the low / high
 *     nibble of byte j+4 below bits 6..7 of byte j-4 / j), 128 bytes of nibbles (weight
 *     64c+i is the low nibble of byte 32c+i, weight 64c+32+i its high nibble);
 *     w = d*sc*q - dmin*m for the weight's 32-wide sub-block.
 *   Q5_K, 176 bytes: the Q4_K header (d, dmin, 12 scale/min bytes), qh[32], then the
 *     Q4_K nibbles; weight 64c+32s+l (s < 2) gains 16 when bit 2c+s of qh[l] is set;
 *     w = d*sc*q - dmin*m with q in 0..31.
 *   Q6_K, 210 bytes: ql[128], qh[64], int8 scales[16], binary16 d; weight 128t+32u+l
 *     (t < 2, u < 4, l < 32) takes its low four bits from the low (u < 2) or high nibble
 *     of ql[64t + 32(u%2) + l] and its top two bits from bits 2u, 2u+1 of qh[32t + l];
 *     w = d * scales[weight/16] * (q - 32).
 *   q4_k_linear / q5_k_linear / q6_k_linear : y[m][n] = x . W^T, W [n][k]
 *   q4_k_/q5_k_/q6_k_linear_fused_gate_up_silu : h = SiLU(x . W_gate^T) * (x . W_up^T), W [2f][k]
 * Arguments, rules and errors as for q8_linear / q8_linear_fused_gate_up_silu (k a
 * positive multiple of 256, the weight base 16-byte aligned).  Two or more rows run the
 * float32 rows kernel in 8-row launches: weights are dequantized exactly in float32 (one
 * fma per weight), one fma per weight and row, and the per-output summation order depends
 * only on k, so those rows are bit-identical whatever m is.  One row runs the one-row
 * kernel when k <= 12288 (fused: k <= 8192; Q6_K: k <= 8192 and a multiple of 2048):
 * per 32-wide sub-block (Q6_K: 16-wide group) t = sum q*x, then acc += d*sc*t - dmin*m*sum x
 * (Q6_K: acc += d*s*(t - 32*sum x)), which agrees with the multi-row results to float32
 * reassociation; other one-row calls run the rows kernel.
 */
q8_status q4_k_linear(const void* w_q4_k, int64_t n, int64_t k,
                      const float* x, int64_t m, int64_t ldx,
                      float* y, int64_t ldy, void* stream);
q8_status q4_k_linear_fused_gate_up_silu(const void* w_gate_up_q4_k, int64_t f, int64_t k,
                                         const float* x, int64_t m, int64_t ldx,
                                         float* h, int64_t ldh, void* stream);
q8_status q5_k_linear(const void* w_q5_k, int64_t n, int64_t k,
                      const float* x, int64_t m, int64_t ldx,
                      float* y, int64_t ldy, void* stream);
q8_status q5_k_linear_fused_gate_up_silu(const void* w_gate_up_q5_k, int64_t f, int64_t k,
                                         const float* x, int64_t m, int64_t ldx,
                                         float* h, int64_t ldh, void* stream);
q8_status q6_k_linear(const void* w_q6_k, int64_t n, int64_t k,
                      const float* x, int64_t m, int64_t ldx,
                      float* y, int64_t ldy, void* stream);
q8_status q6_k_linear_fused_gate_up_silu(const void* w_gate_up_q6_k, int64_t f, int64_t k,
                                         const float* x, int64_t m, int64_t ldx,
                                         float* h, int64_t ldh, void* stream);

/*
 * Integer q8 x q8 path.  The DGX Spark README (Features; Architecture) names GEMV kernels
 * that read Q8_0 directly through int8 dot products, and the qwen3 runner README (q8_0 KV
 * cache; --cache-type) names an integer q8 x q8 dot path over quantized blocks.  No page
 * defines the activation code; the one used here:
 *   per block of 32 inputs, amax = max |x|;  dx = amax / 127;
 *   q = round-half-even(x * (127 / amax)) clamped to [-127, 127],
 *   each quotient and the product rounded to float32 (IEEE, subnormals kept);
 *   a block with amax < 2^-120 (an all-zero block among them) gets dx = 0 and q = 0.
 * Inputs must be finite (a NaN or infinity gives unspecified codes, never a fault).
 *
 * q8_quantize_act: codes and scales of float32 activation rows.
 *   x  : float32 [m][ldx], k > 0 a multiple of 256, ldx >= k (multiple of 4)
 *   xq : int8 [m][k] out, contiguous (row stride k bytes)
 *   xd : float32 [m][k/32] out, contiguous (row stride k/32)
 * x, xq and xd 16-byte aligned.  The result is bit-exact (a pure function of x).
 */
q8_status q8_quantize_act(const float* x, int64_t m, int64_t k, int64_t ldx,
                          int8_t* xq, float* xd, void* stream);

/*
 * y[t][n] = sum over blocks b of (d_w[n][b] * xd[t][b]) * sum_i q_w[n][b][i] * xq[t][b][i]
 * -- the packed-weight linear on int8 activation codes (any int8 value is accepted and
 * multiplied exactly; q8_quantize_act produces [-127, 127]).
 *   w_q8 : Q8_0 [n][k]     xq : int8 [m][k] contiguous     xd : float32 [m][k/32] contiguous
 *   y : float32 [m][ldy], ldy >= n
 * xq and xd 16-byte aligned; other rules as for q8_linear.  Block dot products are exact
 * 32-bit integers; per output, acc = fma(d_w * dx, float(isum), acc) over the blocks in a
 * fixed order that depends only on k, so every row is bit-identical whatever m is.
 */
q8_status q8_linear_q8act(const void* w_q8, int64_t n, int64_t k,
                          const int8_t* xq, const float* xd, int64_t m,
                          float* y, int64_t ldy, void* stream);

/* SiLU(gate) * up from one fused gate_up matrix [2f][k] on int8 activation codes (the
 * fused SwiGLU of q8_linear_fused_gate_up_silu with the arithmetic of q8_linear_q8act). */
q8_status q8_linear_fused_gate_up_silu_q8act(const void* w_gate_up_q8, int64_t f, int64_t k,
                                             const int8_t* xq, const float* xd, int64_t m,
                                             float* h, int64_t ldh, void* stream);

/*
 * Softmax top-k routing (section 14.2: routerTopK with normalize_selected =
 * norm_topk_prob, run on the device here instead of on the host).
 *   x        : float32 [m][ldx], hidden size h (h > 0 a multiple of 256, ldx >= h)
 *   w_router : float32 [n_exp][h], row-major, 1 <= n_exp <= 256
 *   k        : 1 <= k <= n_exp experts per token
 *   normalize: nonzero -> the chosen probabilities are divided by their sum
 *   topk_idx : int32 [m][k] out, descending probability, ties to the lower expert index
 *   topk_w   : float32 [m][k] out
 * Logits and the softmax are computed in float32.
 */
q8_status moe_route_topk(const float* x, int64_t m, int64_t h, int64_t ldx,
                         const float* w_router, int64_t n_exp, int32_t k, int32_t normalize,
                         int32_t* topk_idx, float* topk_w, void* stream);

/*
 * Softmax top-k routing followed by adaptive expert top-p (section 14.2 Config:
 * moe_expert_top_p, 1.0 = full top-k; applyExpertTopP).  The pages give only the knob
 * and its neutral value; the cut used here: with the chosen probabilities p_j in
 * selection order, c_j their running float32 sum through slot j and S the sum over all
 * k slots, slot 0 is kept and slot j >= 1 while c_{j-1} < top_p * S; top_p = 1 keeps
 * all k (and then equals moe_route_topk bit for bit).  Kept weights are divided by the
 * kept sum when normalize is set; a dropped slot gets topk_idx = -1 and topk_w = 0,
 * which q8_moe_grouped_linear skips.
 *   top_p : in (0, 1], else Q8_ERR_SHAPE; other arguments as for moe_route_topk.
 */
q8_status moe_route_topk_top_p(const float* x, int64_t m, int64_t h, int64_t ldx,
                               const float* w_router, int64_t n_exp, int32_t k, int32_t normalize,
                               float top_p, int32_t* topk_idx, float* topk_w, void* stream);

/* Workspace bytes moe_route_topk_ws needs for m tokens and n_exp experts (0 on invalid sizes). */
size_t moe_route_workspace_bytes(int64_t m, int64_t n_exp);

/*
 * moe_route_topk_top_p in two passes that spread each token's logits over many CUs (one
 * kernel block per token is bound by one CU's load rate for the whole router matrix):
 * the logits go to the workspace, then one wave per token selects.  The logits are
 * summed in the same order as in the one-pass calls, so the results are bit-identical
 * to moe_route_topk_top_p (and to moe_route_topk when top_p = 1).
 *   workspace : device memory of at least moe_route_workspace_bytes(m, n_exp) bytes,
 *               16-byte aligned (Q8_ERR_WORKSPACE / Q8_ERR_ALIGN otherwise); its contents
 *               on entry do not matter and are overwritten.
 * Other arguments as for moe_route_topk_top_p.
 */
q8_status moe_route_topk_ws(const float* x, int64_t m, int64_t h, int64_t ldx,
                            const float* w_router, int64_t n_exp, int32_t k, int32_t normalize,
                            float top_p, int32_t* topk_idx, float* topk_w,
                            void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes q8_moe_grouped_linear needs for these sizes (0 on invalid sizes). */
size_t q8_moe_workspace_bytes(int64_t m, int32_t k, int64_t n_exp, int64_t f, int64_t h);

/*
 * Router-weighted SwiGLU expert mixture (section 14.2: moeSwiGluFfnSeq; section 14.4:
 * counting-sort route plan, fixed per-token summation order):
 *   y[t] = sum_{j=0..k-1} topk_w[t][j] * W_down[e] . (SiLU(W_gate[e] x_t) * (W_up[e] x_t)),
 *   e = topk_idx[t][j], summed in slot order j = 0, 1, ..., k-1.
 *   w_gate_up_exps : Q8_0 [n_exp][2f][h] (gate rows [0,f), up rows [f,2f) per expert)
 *   w_down_exps    : Q8_0 [n_exp][h][f]
 *   x : float32 [m][ldx] (ldx >= h)     y : float32 [m][ldy] (ldy >= h)
 *   topk_idx : int32 [m][k], entries in [0, n_exp), or -1 for a slot dropped by
 *              moe_route_topk_top_p (skipped: it contributes nothing; any other entry
 *              outside [0, n_exp) is skipped the same way, but is a caller error)
 *   topk_w   : float32 [m][k]
 *   workspace: device memory of at least q8_moe_workspace_bytes(m, k, n_exp, f, h)
 *              bytes, 256-byte aligned; its contents on entry do not matter.
 * Paths: below 8 routed pairs per expert on average (decode) the float32 GEMV passes run,
 * one pass over an expert's weights serving up to 4 of its routed tokens (an expert with
 * more tokens is streamed again for each further group of 4); from 8 pairs per expert on
 * average the bf16 matrix-core tiles run (activations, d*q and the hidden SiLU*up rounded
 * to bf16 once, float32 accumulation), one pass per 128 of an expert's tokens.  The
 * switch point is the measured crossover on the Qwen3-30B-A3B layer.
 */
q8_status q8_moe_grouped_linear(const void* w_gate_up_exps, const void* w_down_exps,
                                int64_t n_exp, int64_t f, int64_t h,
                                const float* x, int64_t m, int64_t ldx,
                                const int32_t* topk_idx, const float* topk_w, int32_t k,
                                float* y, int64_t ldy,
                                void* workspace, size_t workspace_bytes, void* stream);

/*
 * q8_moe_grouped_linear without a workspace argument and without any allocation, for
 * callers that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid allocation.  The route plan and hidden
 * activations live in a fixed scratch array in device memory that the library holds
 * per device for the life of the process (Q8_MOE_NOALLOC_SCRATCH_BYTES, 16 MiB; about
 * 1170 routed (token, slot) pairs at the Qwen3-30B-A3B sizes f = 768, h = 2048).
 *   Arguments, arithmetic and results as q8_moe_grouped_linear (bit-identical outputs).
 *   Sizes whose workspace (q8_moe_workspace_bytes) exceeds the scratch are refused with
 *   Q8_ERR_WORKSPACE before anything is enqueued.  The first call on a device looks up
 *   the scratch's device address (a runtime query, no allocation).
 *   Every call on one device shares that device's scratch: calls that can overlap on one
 *   device (different streams, different host threads) race and must be serialized by
 *   the caller.  Nothing in the scratch needs to start at any value.
 */
#define Q8_MOE_NOALLOC_SCRATCH_BYTES (16u << 20)
q8_status q8_moe_grouped_linear_noalloc(const void* w_gate_up_exps, const void* w_down_exps,
                                        int64_t n_exp, int64_t f, int64_t h,
                                        const float* x, int64_t m, int64_t ldx,
                                        const int32_t* topk_idx, const float* topk_w, int32_t k,
                                        float* y, int64_t ldy, void* stream);

/*
 * Low-rank adapters of many requests beside a shared packed projection.  Every
 * activation row t may name one adapter a = adapter[t] of a stack; its correction
 *   D[t][i] = scale[a] * sum_{j < r_a} B[a][i][j] * (sum_c A[a][s(i) * rank + j][c] x[t][c])
 * is added to output i of the shared product.  A fused matrix (q/k/v, gate/up) keeps the
 * adapters of its parts apart: its rows are n_sections consecutive sections, and row i
 * uses the `rank` rows of A that belong to its section s(i).
 *   a            : [n_adapters][n_sections * rank][k], b : [n_adapters][n][rank], both of
 *                  element type `type`, contiguous, 16-byte aligned
 *   n_adapters   : 0 .. 256 (0: no row is corrected; a and b may then be NULL)
 *   rank         : a multiple of 8 in 8 .. 256 (the stack's padded rank)
 *   n_sections   : 1 .. 4, section_rows[0 .. n_sections) their sizes (>= 0), summing to n
 *                  (the gate_up calls: to 2f)
 *   ranks        : int32 [n_adapters] device, each adapter's own rank r_a, taken as clamped
 *                  to 0 .. rank; entries of A and B at or past it are not used (they may
 *                  hold anything).  NULL: rank for all.
 *   scale        : float32 [n_adapters] device; NULL: 1 for all
 *   adapter      : int32 [m] device; an entry outside 0 .. n_adapters - 1 (-1 by custom)
 *                  leaves its row without a correction
 * The struct is read during the call only.  Types: A and B elements are widened to
 * float32 exactly; both products accumulate in float32.
 */
typedef enum q8_lora_type { Q8_LORA_F32 = 0, Q8_LORA_F16 = 1, Q8_LORA_BF16 = 2 } q8_lora_type;
#define Q8_LORA_MAX_SECTIONS 4
typedef struct q8_lora {
    const void* a;
    const void* b;
    const int32_t* ranks;
    const float* scale;
    const int32_t* adapter;
    int64_t section_rows[Q8_LORA_MAX_SECTIONS];
    int32_t type; /* q8_lora_type */
    int32_t n_adapters;
    int32_t rank;
    int32_t n_sections;
} q8_lora;

/* Workspace bytes of the two packed calls below for m rows and a matrix of n rows (the
 * gate_up call: n = 2f); 0 on invalid sizes.  Of lora, only rank and n_sections count.  From
 * 256 rows on q8_linear_lora (not the gate_up call) takes lora_workspace_bytes(m, lora) as well. */
size_t q8_linear_lora_workspace_bytes(int64_t m, int64_t n, int64_t k, const q8_lora* lora);

/*
 * The packed linears with adapters:
 *   q8_linear_lora                    : y = x . W^T + D,  W = Q8_0 [n][k]
 *   q8_linear_fused_gate_up_silu_lora : h = SiLU(g) * u with [g u] = x . W^T + D, W = Q8_0 [2f][k]
 * Arguments and errors as for q8_linear / q8_linear_fused_gate_up_silu, and m at most 2^22,
 * f at most 2^29 (Q8_ERR_SHAPE otherwise);
 *   workspace : device memory of at least q8_linear_lora_workspace_bytes(...) bytes,
 *               256-byte aligned; its contents on entry do not matter.  Calls that can
 *               overlap (other streams, or captured graphs replayed side by side) need
 *               workspaces of their own.
 * A row of x that holds a NaN or an infinity gives outputs that are not finite; other rows
 * are not touched by it.  Below 256 rows the arithmetic is of float32 accuracy: products
 * accumulate in float32, and from two rows on (k <= 16384, W below 2 GiB) an element of x is
 * taken to within 2^-30 of its row's largest magnitude (an element below 2^-6 of it so keeps fewer
 * than float32's 24 bits), and a row's outputs have the same bits whatever other rows share the
 * call (their order of summation goes by k, above 4096 also by n and the device).  Beyond that k
 * or size the correction is lora_add's.  From 256 rows on the shared product takes the bf16
 * matrix-core tiles of q8_linear, the correction is lora_add's.  From about 128 rows of rank 64
 * on, the call without adapters followed by lora_add is faster than the call with them.
 */
q8_status q8_linear_lora(const void* w_q8, int64_t n, int64_t k, const float* x, int64_t m, int64_t ldx,
                         const q8_lora* lora, float* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                         void* stream);
q8_status q8_linear_fused_gate_up_silu_lora(const void* w_gate_up_q8, int64_t f, int64_t k, const float* x,
                                            int64_t m, int64_t ldx, const q8_lora* lora, float* h, int64_t ldh,
                                            void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes of lora_add and lora_gate_up_silu for m rows (0 on invalid sizes). */
size_t lora_workspace_bytes(int64_t m, const q8_lora* lora);

/*
 * The adapters alone, beside a shared product of any format that has been computed:
 *   lora_add          : out[t][i] = y[t][i] + D[t][i],  i < n
 *   lora_gate_up_silu : h[t][j] = SiLU(g) * u with g = gu[t][j] + D[t][j], u = gu[t][f + j] + D[t][f + j], j < f
 *   y  : float32 [m][ldy], gu : float32 [m][ldgu] (ldgu >= 2f), 4-byte aligned
 *   x  : float32 [m][ldx], the projection's input (rules as for q8_linear)
 *   out may be y itself (same pointer and leading dimension); otherwise the outputs must
 *   not overlap the inputs.
 *   workspace : at least lora_workspace_bytes(m, lora) bytes, rules as above; m at most 2^22.
 * Float32 accuracy at any m.  Calls whose rows read much of their adapters (48 rows and more,
 * 160 MB together) run on the bf16 matrix cores with every float32 value as three bf16 parts.
 * There nothing of a product is left out for bf16 elements of A and B; for others up to 2^-22
 * (binary16) or 2^-21 (float32) of it, on average the size of a float32 rounding.
 */
q8_status lora_add(const float* y, int64_t n, int64_t ldy, const float* x, int64_t m, int64_t k, int64_t ldx,
                   const q8_lora* lora, float* out, int64_t ldo, void* workspace, size_t workspace_bytes,
                   void* stream);
q8_status lora_gate_up_silu(const float* gu, int64_t f, int64_t ldgu, const float* x, int64_t m, int64_t k,
                            int64_t ldx, const q8_lora* lora, float* h, int64_t ldh, void* workspace,
                            size_t workspace_bytes, void* stream);

/* Workspace bytes q8_moe_layer needs for these sizes (0 on invalid sizes). */
size_t q8_moe_layer_workspace_bytes(int64_t m, int32_t k, int64_t n_exp, int64_t f, int64_t h);

/*
 * The whole mixture-of-experts layer: softmax top-k routing of x (as moe_route_topk_top_p:
 * the same experts, order and weights, bit for bit) followed by the expert mixture (as
 * q8_moe_grouped_linear) of the chosen experts.
 *   w_router, k, normalize, top_p : as for moe_route_topk_top_p (top_p = 1: plain top-k)
 *   w_gate_up_exps, w_down_exps, n_exp, f, h, x, m, ldx, y, ldy : as for q8_moe_grouped_linear
 *   workspace : device memory of at least q8_moe_layer_workspace_bytes(m, k, n_exp, f, h)
 *               bytes, 256-byte aligned; its contents on entry do not matter.  Calls that
 *               can overlap need workspaces of their own.
 * A token whose router probabilities are not finite (a NaN or an infinity in its row)
 * gets NaN in every output; other tokens are not touched by it.  Below 8 routed pairs per
 * expert on average (m * k < 8 * n_exp) the results are of float32 accuracy; from there on
 * the expert products run on the bf16 tiles of q8_moe_grouped_linear.  Up to 128 tokens, 64
 * experts a token and f, h <= 6144 the former is two launches, which take an element of x (and
 * of an expert's hidden row) to within 2^-30 of its row's largest magnitude (below 2^-6 of it
 * that is fewer than float32's 24 bits); a token's outputs then have the same bits whatever
 * other tokens share the call.
 */
q8_status q8_moe_layer(const float* w_router, const void* w_gate_up_exps, const void* w_down_exps, int64_t n_exp,
                       int64_t f, int64_t h, const float* x, int64_t m, int64_t ldx, int32_t k, int32_t normalize,
                       float top_p, float* y, int64_t ldy, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Block-scaled 8-bit floating point.  The DGX Spark README (Performance) serves checkpoints
 * whose weights are FP8 blocks; the pages name the format without spelling it out.  Here:
 *   codes  : OCP e4m3 (1 sign, 4 exponent, 3 fraction bits, bias 7, largest 448, no infinity,
 *            0x7F and 0xFF are NaN), row-major and contiguous, k a positive multiple of 16
 *   scales : float32, contiguous; value = code * scale.  Of a weight matrix [n][k] one scale for
 *            every block of 128 rows x 128 inputs, [ceil(n/128)][ceil(k/128)]; of activations
 *            [m][k] one for every 128 inputs of a row, [m][ceil(k/128)].  The last blocks of
 *            either direction may be cut short.  A fused gate_up matrix [2f][k] is two matrices
 *            of f rows with blocks of their own: its scales are [2 * ceil(f/128)][ceil(k/128)],
 *            gate's first.
 *   type   : of the float operand or result of a call, q8_float_type
 * Sizes: k and the rows of a matrix (n, or 2f) at most 2^20, m at most 2^24, each of m * n, m * k and
 * n * k (n = 2f) at most 2^37; leading dimensions at most 2^30; otherwise Q8_ERR_SHAPE.  Codes 16-byte aligned, scales
 * 4-byte, float operands to their element where nothing else is said; otherwise Q8_ERR_ALIGN.
 * m = 0 and n = 0 (f = 0) enqueue nothing, but that a backward call writes the zeros that an empty
 * sum gives (dw for m = 0, dx for n = 0).  Outputs overlap no input of their call.
 * NaN codes and scales that are not finite give outputs that are not finite where they take
 * part (a row of x: its row; a block of W: its outputs), and nowhere else.
 */
typedef enum q8_float_type { Q8_F32 = 0, Q8_F16 = 1, Q8_BF16 = 2 } q8_float_type;

/*
 * Codes and scales of float rows (blocks of 1 x 128) or of a matrix (blocks of 128 x 128).
 * Of a block's largest magnitude a:
 *   pow2 = 0 : scale = a / 448, code = e4m3(clamp(x * (448 / a), -448, 448))
 *   pow2 = 1 : scale = the least power of two that is at least a / 448, code = e4m3(x / scale)
 * Quotients and products are rounded to float32 once each, codes to nearest even: the result is
 * bit-exact.  a < 2^-116: scale 0 and codes zeros of their elements' signs.  A block that holds a NaN or
 * an infinity: codes and scale NaN.
 *   x : [m][ldx] (w: [n][ldw]) of element type `type`, 16-byte aligned with rows of a multiple of
 *       16 bytes (Q8_ERR_ALIGN otherwise)
 *   q : codes out [m][k]     d : scales out (above)
 */
q8_status f8_quantize_act(const void* x, int32_t type, int64_t m, int64_t k, int64_t ldx, int32_t pow2, uint8_t* q,
                          float* d, void* stream);
q8_status f8_quantize_weight(const void* w, int32_t type, int64_t n, int64_t k, int64_t ldw, int32_t pow2, uint8_t* q,
                             float* d, void* stream);

/*
 * y[t][j] = sum over blocks b of xd[t][b] * wd[j/128][b] * sum_{i in b} xq[t][i] * wq[j][i]
 *   wq, wd : codes [n][k], scales      xq, xd : codes [m][k], scales
 *   y      : [m][ldy] out, element type `type`, ldy >= n
 * acc += (xd * wd) * sum in float32 over the blocks, one rounding to `type` at the end.  With 16-bit
 * results a block's sum runs on the 8-bit matrix cores, which cut a product off at 2^-13 of the largest
 * of the eight that they add at once.  Sums of random codes are off by 2e-5 of their size, whatever k, a
 * tenth of a binary16 result's rounding; a sum whose eights each have one product that is far above the
 * others by up to 2^-10 of the products' magnitudes, which is more than binary16's half step (2^-11), and may
 * be all that is left where the large products cancel.  Results of float32 run on the bf16 matrix cores and
 * are of float32 accuracy whatever the codes.  For one m the order of every sum is fixed by the sizes; it is
 * not the same for every m.
 */
q8_status f8_linear(const uint8_t* wq, const float* wd, int64_t n, int64_t k, const uint8_t* xq, const float* xd,
                    int64_t m, void* y, int32_t type, int64_t ldy, void* stream);

/*
 * h = SiLU(g) * u with [g u] = x . W^T, W = [2f][k] with gate rows first (scales: above), in one
 * launch; SiLU(g) = g / (1 + exp(-g)).
 *   h  : [m][ldh] out, element type `type`, ldh >= f
 *   gu : NULL, or [m][ldgu] out of the same type, ldgu >= 2f: the gate products in columns 0 ..
 *        f - 1, the up products in f .. 2f - 1, as the backward call takes them
 */
q8_status f8_linear_fused_gate_up_silu(const uint8_t* wq, const float* wd, int64_t f, int64_t k, const uint8_t* xq,
                                       const float* xd, int64_t m, void* h, int32_t type, int64_t ldh, void* gu,
                                       int64_t ldgu, void* stream);

/* Workspace bytes of the two backward calls for these sizes (n and f as the calls take them: the
 * fused matrix has 2f rows; 0 on invalid sizes). */
size_t f8_linear_backward_workspace_bytes(int64_t m, int64_t n, int64_t k, int32_t type);
size_t f8_linear_fused_gate_up_silu_backward_workspace_bytes(int64_t m, int64_t f, int64_t k, int32_t type);

/*
 * The gradients of f8_linear's inputs, the quantizers passed straight through:
 *   dx[t][i] = sum_j dy[t][j] * W[j][i]         dw[j][i] = sum_t dy[t][j] * x[t][i]
 * with W and x the values that the codes and scales stand for.
 *   dy : [m][lddy] of element type `type`, lddy >= n
 *   dx : NULL, or [m][lddx] out of that type, lddx >= k
 *   dw : NULL, or [n][lddw] out of that type, lddw >= k (xq, xd: NULL is allowed without it)
 *   workspace : device memory of at least f8_linear_backward_workspace_bytes(...) bytes, 256-byte
 *               aligned; its contents on entry do not matter.  Calls that can overlap need
 *               workspaces of their own.
 * Products run on the bf16 matrix cores with float32 accumulation and one rounding at the end.
 * Codes are exact in bf16.  Gradients of bf16 are taken as they are, binary16 ones as two bf16
 * parts and float32 ones as three, exactly (of float32 numbers below 2^-110 what lies below bf16's least,
 * 2^-133, is left out); a value of x (code * scale) enters dw as two
 * such parts, to within 2^-17, and with float32 gradients as three, exactly as a float32.  Of the products of
 * parts those below 2^-16 (binary16) and 2^-24 (float32) of the whole are left out.
 */
q8_status f8_linear_backward(const uint8_t* wq, const float* wd, int64_t n, int64_t k, const uint8_t* xq,
                             const float* xd, int64_t m, const void* dy, int32_t type, int64_t lddy, void* dx,
                             int64_t lddx, void* dw, int64_t lddw, void* workspace, size_t workspace_bytes,
                             void* stream);

/*
 * The gradients of f8_linear_fused_gate_up_silu's inputs from dh and the gate and up products
 * that it kept.  With s = 1 / (1 + exp(-g)):
 *   dg = dh * u * s * (1 + g * (1 - s)),  du = dh * g * s,  in float32;
 *   dx = [dg du] . W          dw = [dg du]^T . x
 * dg and du enter the products as as many bf16 parts as f8_linear_backward takes gradients of `type`
 * as: rounded to bf16 with bf16, to within 2^-17 with binary16, exactly with float32.
 *   gu : [m][ldgu], ldgu >= 2f;  dh : [m][lddh], lddh >= f, both of element type `type`
 *   dx : NULL, or [m][lddx] out, lddx >= k;  dw : NULL, or [2f][lddw] out, lddw >= k
 * Arithmetic, workspace (f8_linear_fused_gate_up_silu_backward_workspace_bytes) and rules as for
 * f8_linear_backward.
 */
q8_status f8_linear_fused_gate_up_silu_backward(const uint8_t* wq, const float* wd, int64_t f, int64_t k,
                                                const uint8_t* xq, const float* xd, int64_t m, const void* gu,
                                                int64_t ldgu, const void* dh, int32_t type, int64_t lddh, void* dx,
                                                int64_t lddx, void* dw, int64_t lddw, void* workspace,
                                                size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* Q8_LINEAR_H */
