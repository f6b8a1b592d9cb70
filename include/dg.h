/*
 * dg.h -- C ABI of libdg, an FP8 (E4M3 / E5M2) block-scaled NT GEMM for AMD Instinct
 * MI355X (gfx950) with BF16 output, in a dense form and two MoE grouped forms.
 *
 * What every call computes (for each written output element):
 *
 *   C[m,n] = bf16( sum_kb  sA[m,kb] * sB_g[n/128, kb] *
 *                  sum_{k = 128kb}^{128kb+127}  A[m,k] * B_g[n,k] )
 *
 * The operation and its conventions come from the DeepGEMM pages:
 *   - FP8 inputs, BF16 output; the call names gemm_fp8_fp8_bf16_nt,
 *     m_grouped_gemm_fp8_fp8_bf16_nt_contiguous and ..._masked, and the alignment
 *     query get_m_alignment_for_contiguous_layout: aisharenet.com/ja usage guide,
 *     sections 1-3 of "main functions".
 *   - NT layout only (LHS not transposed, RHS transposed, i.e. B stored N x K); casting
 *     and transposition are the caller's job: turtlesai.it summary, technical paragraph.
 *   - fine-grained scaling and two-level accumulation: same paragraph, and the
 *     chattools.cn article, section on core design ideas.  Each 128-deep K block's
 *     product is formed on its own, multiplied by sA*sB and added into a separate fp32
 *     accumulator; the result is rounded to bf16 with round-to-nearest-even.
 *   - grouping on the M axis only, every group sharing N and K: aisharenet.com/ja usage
 *     guide, section 2; contiguous layout for training / prefill and masked layout for
 *     decode, usable under graph capture: flashmla.org/zh page, section "DeepGEMM
 *     performance".
 *
 * Conventions shared by every call:
 *   - Memory: every pointer is a DEVICE pointer owned by the caller.  The library
 *     allocates and frees nothing.  C is an output the library writes in place.
 *     Pointers and stream belong to the current device, on which the call launches.
 *   - Layouts (all row-major, densely packed):
 *       A  e4m3fn bytes,   rows x K         sA fp32, rows x (K/128)
 *       B  e4m3fn bytes,   G x N x K        sB fp32, G x ceil(N/128) x (K/128)
 *       C  bf16 bits,      rows x N
 *     e4m3fn is the OCP 8-bit format E4M3 (bias 7, max 448, no infinities, NaN = S.1111.111);
 *     the _ex calls also take E5M2 for either operand.
 *     Column n of C uses row n/128 of its group's sB; N need not be a multiple of 128.
 *   - Preconditions checked on the host, before any device work, in this order:
 *       shapes: 0 < K <= 2^22 and K % 128 == 0, M/N >= 0, G >= 1,
 *       cap >= 0, fewer than 2^31 64x64 output tiles              -> DG_ERR_SHAPE
 *       operand formats (the _ex calls) DG_FP8_E4M3 or DG_FP8_E5M2  -> DG_ERR_FORMAT
 *       an empty output (no rows or N == 0) returns DG_OK without touching anything
 *       pointers non-NULL                                         -> DG_ERR_NULL
 *       A, B, C 16-byte aligned; sA, sB, group_idx, masked_m 4-byte -> DG_ERR_ALIGN
 *       workspace_bytes >= dg_workspace_bytes(...) and workspace
 *       non-NULL when that is > 0                                 -> DG_ERR_WORKSPACE
 *       current device is a gfx950 GPU                            -> DG_ERR_DEVICE
 *     A failed launch returns DG_ERR_HIP.  Values that live in device memory
 *     (group_idx, masked_m) are never read on the host; their rules are stated per call.
 *   - Execution: every call is asynchronous on `stream` (a hipStream_t; NULL is the
 *     null stream), never synchronises, and performs no host readback, so it may be
 *     captured in a HIP graph.  Faults inside kernels surface at the caller's next
 *     synchronisation.  Results are deterministic: the same inputs give the same bits.
 *   - Range: each K block's partial, the factor sA*sB and the accumulator are fp32, so a
 *     result is exact up to fp32 rounding as long as they stay inside the fp32 range.
 *     Scales from the quantisation calls below keep sA*sB finite whenever the two
 *     blocks' maxima multiply to less than about 6.8e43 (448^2 * FLT_MAX); beyond that
 *     the factor is +inf and the element becomes +-inf or NaN (0 * inf, inf - inf).
 *   - Workspace: device memory the caller lends for split-K partial sums, at least
 *     dg_workspace_bytes(...) bytes, 16-byte aligned.  It must be zero filled before
 *     its first use; every call leaves it zero filled again (a zero word marks a partial
 *     not yet written), so one workspace can serve calls of any shape in stream order.
 *     Two calls that may run concurrently must not share one workspace.
 *   - Split-K calls (those with a workspace) never depend on one another's workgroups
 *     making progress: the workgroups sharing an output tile reduce it together when
 *     they all run at once, and the last of them to finish its share completes whatever
 *     is left, summing the tile's partials in a fixed order.  So the result does not
 *     depend on scheduling or on other work sharing the GPU.
 */
#ifndef DG_H_
#define DG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int dg_status;
#define DG_OK 0
#define DG_ERR_NULL 1
#define DG_ERR_SHAPE 2
#define DG_ERR_ALIGN 3
#define DG_ERR_WORKSPACE 4
#define DG_ERR_DEVICE 5
#define DG_ERR_HIP 6
#define DG_ERR_FORMAT 7

/* 8-bit operand formats (OCP): E4M3 ("fn": bias 7, max 448, no infinities) and E5M2
 * (bias 15, max 57344, with infinities).  The usage guide allows either for the inputs
 * (aisharenet.com/ja usage guide, main functions, section 1). */
#define DG_FP8_E4M3 0
#define DG_FP8_E5M2 1

#define DG_DENSE 0
#define DG_CONTIGUOUS 1
#define DG_MASKED 2

/* Row alignment that each group's segment must have in the contiguous layout
 * (aisharenet.com/ja usage guide, section 2: group sizes aligned to the GEMM M block).
 * Returns 128. */
int dg_get_m_alignment_for_contiguous_layout(void);

/* Static, human-readable name of a status code ("DG_OK", ...); never NULL. */
const char *dg_status_string(dg_status status);

/* Workspace bytes the call of kind `kind` (DG_DENSE / DG_CONTIGUOUS / DG_MASKED) needs
 * for these sizes; rows_or_cap is M, M_total or cap.  0 when none is needed.  Returns
 * 0 for invalid shapes (the call itself then reports DG_ERR_SHAPE). */
size_t dg_workspace_bytes(int kind, int64_t rows_or_cap, int64_t N, int64_t K, int64_t G);

/* Name of the kernel instance the call of kind `kind` would use for these sizes
 * (a static string), or "none" for invalid or empty shapes.  Host-only; for logging
 * and tests. */
const char *dg_instance_name(int kind, int64_t rows_or_cap, int64_t N, int64_t K, int64_t G);

/* Dense NT GEMM: C (M x N) = A (M x K) x B (N x K)^T with sA (M x K/128) and
 * sB (ceil(N/128) x K/128).  Every element of C is written.
 * (aisharenet.com/ja usage guide, section 1: gemm_fp8_fp8_bf16_nt.) */
dg_status dg_gemm_fp8_nt(const uint8_t *A, const float *sA,
                         const uint8_t *B, const float *sB,
                         uint16_t *C, int64_t M, int64_t N, int64_t K,
                         void *workspace, size_t workspace_bytes, void *stream);

/* Contiguous grouped NT GEMM (MoE training forward / prefill).  The rows of all groups
 * are concatenated into A (M_total x K); B holds G matrices N x K back to back.
 * group_idx (DEVICE, M_total int32) names the group of each row.  Segments are
 * expected to be 128-row aligned (dg_get_m_alignment_for_contiguous_layout); the
 * defined rule for any content is: row m is written with B[group_idx[m]] iff
 * 0 <= group_idx[m] < G and group_idx[m] == group_idx[128*floor(m/128)]; every other
 * row of C is left untouched (so -1 can mark padding rows).  Segments may come in any
 * group order.  (aisharenet.com/ja usage guide, section 2.) */
dg_status dg_grouped_gemm_fp8_contiguous(const uint8_t *A, const float *sA,
                                         const uint8_t *B, const float *sB,
                                         const int32_t *group_idx, uint16_t *C,
                                         int64_t M_total, int64_t N, int64_t K, int64_t G,
                                         void *workspace, size_t workspace_bytes,
                                         void *stream);

/* Masked grouped NT GEMM (MoE decode).  A is G x cap x K (sA G x cap x K/128), B is
 * G x N x K, C is G x cap x N.  masked_m (DEVICE, G int32) gives each group's count of
 * valid leading rows, clamped to [0, cap] on the device; group g writes rows
 * [0, masked_m[g]) of its C block and never writes the others, and A rows at or past
 * masked_m[g] are never read (they may hold anything).  Nothing is read back to the
 * host, so the call can be captured once and replayed with new counts.
 * (aisharenet.com/ja usage guide, section 3; flashmla.org/zh, "DeepGEMM performance".) */
dg_status dg_grouped_gemm_fp8_masked(const uint8_t *A, const float *sA,
                                     const uint8_t *B, const float *sB,
                                     const int32_t *masked_m, uint16_t *C,
                                     int64_t G, int64_t cap, int64_t N, int64_t K,
                                     void *workspace, size_t workspace_bytes, void *stream);

/* dg_gemm_fp8_nt for callers that cannot allocate device memory (code under graph
 * capture, serving loops that must not call hipMalloc): no workspace argument and no
 * allocation of any kind.  Split-K calls use instead a workspace the library holds in a
 * statically sized device array, one per GPU, kept until the process ends: at most
 * 32 MiB + 64 KiB (enough for every shape this library accepts; a shape needing more
 * would return DG_ERR_WORKSPACE).  On the first call for a device the array's address
 * is looked up and, unless `stream` is being captured, the array is zeroed by a kernel
 * on `stream` (make that first call outside graph capture); every call leaves it zero
 * filled.  All calls on one GPU share the array:
 * two such calls that may overlap in time (on different streams, or from different
 * host threads without ordering) race and give undefined results; calls in one stream's
 * order are fine.  Otherwise as dg_gemm_fp8_nt (E4M3 operands, same errors; DG_ERR_HIP
 * if the array's address cannot be had). */
dg_status dg_gemm_fp8_nt_noalloc(const uint8_t *A, const float *sA,
                                 const uint8_t *B, const float *sB,
                                 uint16_t *C, int64_t M, int64_t N, int64_t K, void *stream);

/* The same three calls with explicit operand formats: a_format / b_format are
 * DG_FP8_E4M3 or DG_FP8_E5M2 (any pair), else DG_ERR_FORMAT.  The calls above are these
 * with both formats DG_FP8_E4M3.  Everything else (layouts, scales, routing, workspace,
 * errors, execution) is as described there; the choice of kernel instance, and hence
 * dg_workspace_bytes / dg_instance_name, does not depend on the formats.
 * (aisharenet.com/ja usage guide, main functions, section 1: E4M3 or E5M2 inputs.) */
dg_status dg_gemm_fp8_nt_ex(const uint8_t *A, int a_format, const float *sA,
                            const uint8_t *B, int b_format, const float *sB,
                            uint16_t *C, int64_t M, int64_t N, int64_t K,
                            void *workspace, size_t workspace_bytes, void *stream);
dg_status dg_grouped_gemm_fp8_contiguous_ex(const uint8_t *A, int a_format, const float *sA,
                                            const uint8_t *B, int b_format, const float *sB,
                                            const int32_t *group_idx, uint16_t *C,
                                            int64_t M_total, int64_t N, int64_t K, int64_t G,
                                            void *workspace, size_t workspace_bytes,
                                            void *stream);
dg_status dg_grouped_gemm_fp8_masked_ex(const uint8_t *A, int a_format, const float *sA,
                                        const uint8_t *B, int b_format, const float *sB,
                                        const int32_t *masked_m, uint16_t *C,
                                        int64_t G, int64_t cap, int64_t N, int64_t K,
                                        void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------
 * fp8 quantisation with block scales: the casting step in front of the GEMM, which the
 * pages leave to the caller (turtlesai.it summary, technical paragraph), in the two
 * block shapes of the method's fine-grained scaling (chattools.cn, core design ideas):
 * one scale per 1x128 block of a row (activations, the sA layout) and one per 128x128
 * block (weights, the sB layout).
 *
 * Per block: amax = max |x| in fp32; scale = amax / FMAX in fp32 (FMAX = 448 for E4M3,
 * 57344 for E5M2; 1 for an all-zero block); each code is x / scale, an IEEE fp32
 * division, rounded to the nearest value of `format`, ties to even, saturating at
 * +-FMAX.  So Q * S reproduces X to within half an fp8 step of each block's scale.
 *
 * Inputs: X rows x K (row-major, DEVICE, 16-byte aligned), x_dtype DG_IN_F32 or
 * DG_IN_BF16.  A block that holds a NaN has a NaN scale, one that holds an infinity (and no
 * NaN) an infinite one, and unspecified codes: what uses it comes out infinite or NaN.  K > 0, K % 128 == 0 (DG_ERR_SHAPE); rows >= 0 (0: nothing
 * to do).  Outputs (DEVICE, caller-owned): Q rows x K codes (8-byte aligned); S rows x
 * K/128 (1x128) or ceil(rows/128) x K/128 (128x128) fp32 (4-byte aligned).
 * Errors: DG_ERR_SHAPE, DG_ERR_FORMAT (format or x_dtype), DG_ERR_NULL, DG_ERR_ALIGN,
 * DG_ERR_DEVICE, DG_ERR_HIP, checked in that order.  Asynchronous on `stream`,
 * graph-capturable, deterministic. */
#define DG_IN_F32 0
#define DG_IN_BF16 1

dg_status dg_quantize_fp8_1x128(const void *X, int x_dtype, uint8_t *Q, float *S,
                                int64_t rows, int64_t K, int format, void *stream);
dg_status dg_quantize_fp8_128x128(const void *X, int x_dtype, uint8_t *Q, float *S,
                                  int64_t rows, int64_t K, int format, void *stream);

/* Transposition of a byte matrix (fp8 codes): Y (cols x rows) = X (rows x cols)^T, both
 * row-major DEVICE buffers, 16-byte aligned, rows and cols multiples of 16.  The calls
 * above take the NT layout only and leave transposition to the caller (turtlesai.it
 * summary, technical paragraph); this turns a K x N operand into the N x K one they
 * take.  (Its 128x128 scale matrix transposes as an ordinary small fp32 matrix.)
 * Errors: DG_ERR_SHAPE, DG_ERR_NULL, DG_ERR_ALIGN, DG_ERR_DEVICE, DG_ERR_HIP, in that
 * order; rows or cols 0: nothing to do.  Asynchronous on `stream`. */
dg_status dg_transpose_fp8(const uint8_t *X, uint8_t *Y, int64_t rows, int64_t cols,
                           void *stream);

/* ---------------------------------------------------------------------------------
 * The gate of a mixture of experts: from a row's logits to the experts that the grouped
 * calls above compute for it, and what training needs of that choice.
 *
 * For each row t of the T x E logits z (row-major, DEVICE, row stride ld >= E elements,
 * dtype DG_IN_F32 or DG_IN_BF16), in fp32:
 *   scores   s_te = softmax over e (DG_SCORE_SOFTMAX) or sigmoid of z_te (DG_SCORE_SIGMOID)
 *   choice   ids[t][0..k) = the experts of the k largest keys z_te + bias_e (one fp32
 *            addition; bias NULL: z_te), in decreasing order, equal keys in increasing order
 *            of e.  A key of -inf or NaN is never chosen: a bias of -inf closes an expert;
 *            choices that are left without an expert have id -1 and weight 0.
 *   weights  weights[t][j] = scale * s of the choice, divided, if `normalize` is non-zero,
 *            by the sum of the row's chosen scores.  The quotients keep their precision
 *            however small the scores are (sigmoid: down to about e^-600; scores below count
 *            as 0, and 0 / 0 as 0).  The bias is part of the choice only.  It is added to the
 *            logits: a correction that was trained to be added to the scores, as the gates
 *            with one that keeps the experts balanced have it, orders experts differently,
 *            and no bias on the logits does what it does.
 *   row_valid (T bytes or NULL: all rows): a row of 0 is padding.  Its logits may be
 *            anything; its ids are -1, its weights 0, and it is in no count, loss or gradient.
 * and over the rows:
 *   counts   counts[e] = choices of expert e (the masked call's masked_m, or the contiguous
 *            call's segment lengths before their alignment)
 *   loss     balance * sum_e f_e P_e, f_e = E counts[e] / (k V), P_e = the mean over the V
 *            valid rows of p_te, with p = s (softmax) or s / sum_e s (sigmoid); 0 if V = 0.
 *            Its derivative by p_te, f being a constant, is the same for every valid row:
 *   coef     coef[e] = balance * f_e / V, what the backward pass needs of the loss.
 * A row of -inf only has no choice and no probabilities.  Under softmax a row with a NaN or a
 * +inf has NaN weights; under sigmoid the weights come from the choices' own logits and stay
 * finite, so they do not show a NaN among the others.  A NaN, and under softmax a
 * +inf, makes the loss NaN.  ids stay in range.
 *
 * 1 <= E <= 1024, 1 <= k <= min(E, 16), T >= 0 (T = 0: counts, loss and coef are written as
 * zeros, nothing else).  counts may be NULL; loss and coef are both given or both NULL, and
 * need counts.  Pointers need their element's alignment only (rows that start on 16 bytes,
 * 8 for bf16, with E and ld multiples of 4, are read in wider loads).
 *
 * With counts the call needs a workspace of dg_moe_route_workspace_bytes bytes (0 for a few
 * rows: none), 16-byte aligned.  It may hold anything before and after the call, so one
 * buffer can serve this call and dg_lora_bf16 in stream order, whichever host threads make
 * the calls: what a call launches is enqueued with nothing of another call with the same
 * buffer between (not two calls that may overlap on the GPU, not buffers that overlap in
 * part, and not the GEMM calls, which need theirs zero).
 *
 * Sums over rows are taken in an order that depends on the sizes only: the same inputs give
 * the same bits.  Over several workgroups the loss is added up in multiples of
 * balance * E * 2^-44, at most 64 of them: beside fp32's relative error it has an absolute
 * one of balance * E * 2^-39 at most.
 * Errors, in this order: DG_ERR_SHAPE, DG_ERR_FORMAT (dtype or score), DG_ERR_NULL,
 * DG_ERR_ALIGN, DG_ERR_WORKSPACE, DG_ERR_DEVICE, DG_ERR_HIP.  Asynchronous on `stream`,
 * no readback, graph-capturable. */
#define DG_SCORE_SOFTMAX 0
#define DG_SCORE_SIGMOID 1

size_t dg_moe_route_workspace_bytes(int64_t T, int64_t E);
dg_status dg_moe_route(const void *logits, int dtype, int64_t ld, const float *bias,
                       const uint8_t *row_valid, int64_t T, int64_t E, int64_t k, int score,
                       int normalize, float scale, float balance, int32_t *ids,
                       float *weights, int32_t *counts, float *loss, float *coef,
                       void *workspace, size_t workspace_bytes, void *stream);

/* Backward pass of dg_moe_route: grad_logits (T x E, row stride ld_grad, dtype of the
 * logits; every element is written, padding rows with zeros) = the gradient by the logits of
 *   sum_tj grad_weights[t][j] weights[t][j] + grad_loss * loss
 * with the choice and the counts held constant.  logits, row_valid, score, normalize, scale
 * as in the forward call, ids and coef its outputs.  grad_weights NULL: no first term (ids
 * may then be NULL).  coef NULL: no second term (a NaN of a sigmoid row then stays in its own
 * element); grad_loss (one fp32 in DEVICE memory) NULL
 * with coef: 1.  ids outside [0, E) are skipped; a row's ids must differ from each other.
 * No workspace.  Errors and execution as above. */
dg_status dg_moe_route_backward(const void *logits, int dtype, int64_t ld,
                                const uint8_t *row_valid, int64_t T, int64_t E, int64_t k,
                                int score, int normalize, float scale, const int32_t *ids,
                                const float *grad_weights, const float *coef,
                                const float *grad_loss, void *grad_logits, int64_t ld_grad,
                                void *stream);

/* ---------------------------------------------------------------------------------
 * Low-rank adapters of many requests beside a shared projection (dg_gemm_fp8_nt's output,
 * or any other bf16 matrix, as `base`):
 *
 *   out[t,n] = bf16( base[t,n] + scales[i] * sum_r ( sum_k X[t,k] A_i[r,k] ) B_i[n,r] )
 *
 * with i = ids[t], r < ranks[i].  Rows whose id is outside [0, L) have no adapter: out =
 * base.  All DEVICE, row-major:
 *   X  bf16, T x K, row stride ldx     A  bf16, L x R x K     B  bf16, L x N x R
 *   ids int32, T   scales fp32, L (NULL: 1)   ranks int32, L (NULL: all R; clamped to
 *   [0, R] on the device; what A and B hold past an adapter's rank does not count)
 *   base bf16, T x N, row stride ld_base (NULL: zero; may be `out` itself with the same
 *   stride, not overlap it otherwise)         out bf16, T x N, row stride ld_out
 * Rows of one adapter may be anywhere.  A row's result depends on its own adapter's values
 * only, whatever other adapters hold; an infinity or NaN in it makes the results that it
 * takes part in infinite or NaN.  Sums are fp32; the inner product (times the scale) is kept
 * to 16 significant bits or more, as infinite past bf16's largest number, and the result
 * rounded once, to nearest even.
 *
 * T, N >= 0 (0: nothing to do), K > 0 and K % 128 == 0, N, K <= 2^22, 8 <= R <= 128 and
 * R % 8 == 0, L >= 1, ldx % 8 == 0, strides at least the row's length (DG_ERR_SHAPE).
 * X, A, B 16-byte aligned, base and out 2-byte (faster: 16-byte with strides that 8
 * divides).  Workspace: dg_lora_workspace_bytes bytes, 16-byte aligned; it may hold
 * anything before and after (see dg_moe_route).
 * Errors, in this order: DG_ERR_SHAPE, DG_ERR_NULL, DG_ERR_ALIGN, DG_ERR_WORKSPACE,
 * DG_ERR_DEVICE, DG_ERR_HIP.  Asynchronous on `stream`, graph-capturable, deterministic. */
size_t dg_lora_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t R, int64_t L);
dg_status dg_lora_bf16(const uint16_t *X, int64_t ldx, const uint16_t *A, const uint16_t *B,
                       const int32_t *ids, const float *scales, const int32_t *ranks,
                       const uint16_t *base, int64_t ld_base, uint16_t *out, int64_t ld_out,
                       int64_t T, int64_t N, int64_t K, int64_t R, int64_t L,
                       void *workspace, size_t workspace_bytes, void *stream);

/* ---------------------------------------------------------------------------------
 * A feed-forward block in 8 bits, between and behind the GEMM calls: the norm in front, the
 * gated first half, and the backward passes of both from 8-bit checkpoints.  Codes and
 * scales are everywhere those of dg_quantize_fp8_1x128 (one fp32 scale per 128 columns of a
 * row, amax / FMAX, 1 for a block of zeros; code = value / scale, nearest; a quotient within
 * 2^-22 of itself of the border between two codes may go to either), formed from fp32 values
 * that are rounded nowhere before: the operands of the GEMM calls as they stand.  A block that holds a NaN has a NaN scale; one that holds an
 * infinity (and no NaN) an infinite one.  All pointers are DEVICE pointers, T, rows and
 * M_total may be 0 (nothing is done unless a call says otherwise), everything is
 * asynchronous on `stream`, without readback, deterministic and graph-capturable, and no two
 * buffers of a call may overlap unless a call says so.  Errors, in this order: DG_ERR_SHAPE,
 * DG_ERR_FORMAT (formats, dtypes, activation), DG_ERR_NULL, DG_ERR_ALIGN, DG_ERR_WORKSPACE,
 * DG_ERR_DEVICE, DG_ERR_HIP.
 *
 * Root-mean-square norm of T rows of K, behind the residual's addition:
 *   h = X + residual   (fp32 sum rounded to `dtype`; residual NULL: h = X)
 *   rstd = 1 / sqrt(mean of h^2 over the row + eps),   y = (h rstd) weight
 * X, residual and H of `dtype` (DG_IN_F32 or DG_IN_BF16), weight K of weight_dtype (NULL: 1).
 * Outputs, each NULL if it is not wanted: H (given if and only if residual is; it may be X or
 * residual themselves, with the same stride), codes Q (T x K, dense) with scales S
 * (T x K/128), Y = bf16(y) (its codes come from y, not from Y), rstd (T fp32, for the backward
 * pass).  A row whose h^2 pass the fp32 range has rstd 0; one of zeros, or whose h^2 are
 * below that range, needs eps > 0; a row with a NaN is NaN.
 * 0 < K <= 65536, K % 128 == 0; row strides at least K and multiples of 8 (DG_ERR_SHAPE).
 * X, residual, weight, H, Y 16-byte aligned, Q 8, S and rstd 4. */
dg_status dg_rms_norm_fp8(const void *X, int dtype, int64_t ldx, const void *residual,
                          int64_t ld_residual, const void *weight, int weight_dtype, float eps,
                          void *H, int64_t ldh, uint8_t *Q, float *S, int format, uint16_t *Y,
                          int64_t ldy, float *rstd, int64_t T, int64_t K, void *stream);

/* Backward pass of the norm, H and rstd being the forward call's (H = X without a residual):
 *   g = weight grad_y,  grad_x = rstd (g - h rstd^2 mean(g h)) + grad_h
 *   grad_weight = sum over rows of grad_y h rstd
 * grad_x (dtype) is the gradient by X and by the residual alike; grad_h (dtype, NULL: none) is
 * the gradient that reaches H itself, the residual stream's, and may be grad_x, as grad_y and H
 * may (same stride).  grad_weight (K fp32, NULL: not wanted) is written, with zeros for T = 0; its
 * sums are fp32, in an order that depends on the sizes only.  Shapes and alignments as above.
 * With grad_weight a workspace of dg_rms_norm_backward_workspace_bytes bytes, 16-byte aligned,
 * that may hold anything before and after (see dg_moe_route). */
size_t dg_rms_norm_backward_workspace_bytes(int64_t T, int64_t K);
dg_status dg_rms_norm_backward(const void *grad_y, int dtype, int64_t ld_grad_y, const void *H,
                               int64_t ldh, const float *rstd, const void *weight,
                               int weight_dtype, const void *grad_h, int64_t ld_grad_h,
                               void *grad_x, int64_t ld_grad_x, float *grad_weight, int64_t T,
                               int64_t K, void *workspace, size_t workspace_bytes,
                               void *stream);

/* The first half of a gated feed-forward block in one kernel:
 *   G = A Bg^T,  U = A Bu^T   (block-scaled products as in dg_gemm_fp8_nt, kept in fp32)
 *   h = act(G) U,   act(x) = x sigmoid(x)                                   (DG_ACT_SILU)
 *                   act(x) = x sigmoid(2 sqrt(2/pi) (x + 0.044715 x^3))     (DG_ACT_GELU: the
 *                                                                           tanh form of gelu)
 * out as codes H (rows x N) and scales sH (rows x N/128) of out_format, the A operand of the
 * down projection's call.  A, sA, B, sB, group_idx, masked_m, formats and row rules are those
 * of the GEMM calls, with B (a group's) the gate's N rows and then the up matrix's N, sB their
 * 2N/128 rows of scales.  GU and sGU (both or neither): codes (rows x 2N: gate, then up) and
 * scales (rows x 2N/128) of G and U in out_format, the checkpoint for dg_gated_backward.  Rows
 * that the GEMM call would not write keep what H, sH, GU and sGU held.
 * N % 128 == 0, N <= 2^20, K % 128 == 0, 0 < K <= 2^22.  A, B, H, GU 16-byte aligned, the rest 4.
 * Workspace: dg_gated_workspace_bytes(kind, rows or cap, N, K, G) bytes (0 for many rows), 16-byte
 * aligned, that may hold anything before and after (see dg_moe_route). */
#define DG_ACT_SILU 0
#define DG_ACT_GELU 1

size_t dg_gated_workspace_bytes(int kind, int64_t rows_or_cap, int64_t N, int64_t K, int64_t G);
dg_status dg_gated_fp8_nt(const uint8_t *A, int a_format, const float *sA, const uint8_t *B,
                          int b_format, const float *sB, uint8_t *H, float *sH, int out_format,
                          uint8_t *GU, float *sGU, int activation, int64_t M, int64_t N,
                          int64_t K, void *workspace, size_t workspace_bytes, void *stream);
dg_status dg_grouped_gated_fp8_contiguous(const uint8_t *A, int a_format, const float *sA,
                                          const uint8_t *B, int b_format, const float *sB,
                                          const int32_t *group_idx, uint8_t *H, float *sH,
                                          int out_format, uint8_t *GU, float *sGU,
                                          int activation, int64_t M_total, int64_t N, int64_t K,
                                          int64_t G, void *workspace, size_t workspace_bytes,
                                          void *stream);
dg_status dg_grouped_gated_fp8_masked(const uint8_t *A, int a_format, const float *sA,
                                      const uint8_t *B, int b_format, const float *sB,
                                      const int32_t *masked_m, uint8_t *H, float *sH,
                                      int out_format, int activation, int64_t G, int64_t cap,
                                      int64_t N, int64_t K, void *workspace,
                                      size_t workspace_bytes, void *stream);

/* Backward pass of the gated half up to the gradients by G and U, from the checkpoint:
 *   D = (grad_H u act'(g), grad_H act(g)),  g and u the values that GU and sGU stand for
 * grad_H T x N of dtype (dense), GU and sGU as the forward call wrote them in gu_format; D
 * (T x 2N: by the gate, then by up) and sD (T x 2N/128) in out_format: the A operand of the
 * call that forms the gradient by A (with B transposed, dg_transpose_fp8) and P of the weight
 * gradient.  D and sD may be GU and sGU.  group_idx (T, or NULL: every row) with G as in the
 * contiguous call: rows that it would not write are neither read nor written.
 * N % 128 == 0, N <= 2^20, T N <= 2^35.  grad_H, GU and D 16-byte aligned, the rest 4. */
dg_status dg_gated_backward(const void *grad_H, int dtype, const uint8_t *GU, int gu_format,
                            const float *sGU, const int32_t *group_idx, int activation,
                            uint8_t *D, float *sD, int out_format, int64_t T, int64_t N,
                            int64_t G, void *stream);

/* A weight's gradient from two 8-bit matrices that lie row by row, such as a gradient's codes
 * and an activation's checkpoint:
 *   dW[n,k] = sum over rows t of  (sP[t,n/128] P[t,n]) (sQ[t,k/128] Q[t,k])
 * P T x N, sP T x N/128, Q T x K, sQ T x K/128; dW N x K of dtype, added to if `accumulate` is
 * non-zero, else overwritten.  In the grouped form dW is G x N x K and row t counts for group
 * group_idx[t] by the contiguous call's rule; the others' codes and scales may be anything; a
 * group without rows has a gradient of zeros (T = 0: zeros everywhere).
 * The products' factors are bf16: a code is one, a code with its scales is rounded once to 8
 * bits (exactly kept for scales that are powers of two); sums are fp32, in an order that
 * depends on the sizes only.
 * N, K % 128 == 0, N, K <= 2^22, G (N/128) (K/128) < 2^23.  P, Q, dW 16-byte aligned, the rest 4.
 * Workspace: dg_wgrad_workspace_bytes bytes (G = 1 for the dense form), 16-byte aligned, that
 * may hold anything before and after (see dg_moe_route). */
size_t dg_wgrad_workspace_bytes(int64_t T, int64_t N, int64_t K, int64_t G);
dg_status dg_wgrad_fp8(const uint8_t *P, int p_format, const float *sP, const uint8_t *Q,
                       int q_format, const float *sQ, void *dW, int dtype, int accumulate,
                       int64_t T, int64_t N, int64_t K, void *workspace,
                       size_t workspace_bytes, void *stream);
dg_status dg_grouped_wgrad_fp8_contiguous(const uint8_t *P, int p_format, const float *sP,
                                          const uint8_t *Q, int q_format, const float *sQ,
                                          const int32_t *group_idx, void *dW, int dtype,
                                          int accumulate, int64_t M_total, int64_t N, int64_t K,
                                          int64_t G, void *workspace, size_t workspace_bytes,
                                          void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DG_H_ */
