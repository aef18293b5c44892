/*
 * gba_moe.h -- C ABI of libgba_moe: what stands around the products of a mixture of
 * experts (gba_experts.h) on MI355X (gfx950): routing of tokens to experts, sorting and
 * movement of their rows, and products in 8-bit floating point with a scale for each
 * block of 128, forward and backward. It shares the enums (gba_dtype, gba_act) and status
 * codes of gba.h.
 *
 * Conventions shared by every entry point (as gba_experts.h unless stated):
 *   - All array arguments are DEVICE pointers owned by the caller, dense and
 *     row-major. The library allocates nothing and keeps no pointer after a call.
 *   - 16-bit and 8-bit matrices are 16-byte aligned, with rows of a multiple of 8
 *     values in 16 bits and of 16 in 8 bits; all other arrays have the alignment of their
 *     type: GBA_ERR_ALIGN.
 *   - Argument errors are reported synchronously, before any launch. Work is
 *     enqueued on the calling thread's stream (gbm_set_stream) and runs
 *     asynchronously. Nothing synchronises, allocates or copies, so every entry
 *     point can be recorded in a HIP graph.
 *   - No output may overlap an input, another output or the workspace: GBA_ERR_ALIAS.
 *     Calls that share a workspace must be ordered on one stream.
 *   - Unknown flag bits: GBA_ERR_SHAPE.
 *   - A launch failure returns GBA_ERR_HIP (gbm_last_hip_error() gives the
 *     code); a device that is not gfx950 GBA_ERR_DEVICE.
 *   - Results are the same bits in every run (but for rows that two slots name, see below).
 *
 * Slots and rows. Token t's j-th expert, slot (t, j), is indices[t][j], or -1. Rows are
 * sorted by expert, rows of one expert by (t, j): expert e owns rows offsets[e] ..
 * offsets[e+1] - 1, the groups of gba_experts.h, and rows[t][j] is the row of slot (t, j), or -1.
 * No row belongs to two slots, as moe_sort leaves rows: where a caller's own rows name one twice, calls that write rows
 * (moe_dispatch, dy of moe_combine_grad, fp8_quantize) leave in it, place by place, a value of either slot, in another
 * mixture in another run, and fp8_quantize may leave one slot's codes with the other's scales.
 * T k <= 2^29. Whatever indices and rows hold, nothing outside the arrays is touched: an
 * expert outside [0, E) or a row outside [0, R) counts as -1.
 */
#ifndef GBA_MOE_H
#define GBA_MOE_H

#include "gba.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Stream for this thread's later calls of this library (a hipStream_t). */
int gbm_set_stream(void *hip_stream);
int gbm_last_hip_error(void);
const char *gbm_version(void);

/* ------------------------------------------------------------------ routing -- */

enum { GBM_DTYPE_F32 = 2 };                     /* logits: beside gba_dtype */
enum { GBM_SOFTMAX = 0, GBM_SIGMOID = 1 };      /* score */
enum { GBM_RENORMALIZE = 1 };                   /* flags of moe_route and its gradient */
#define GBM_MAX_ROUTED 1024                     /* experts */
#define GBM_MAX_TOP 32                          /* experts of a token */
#define GBM_MAX_EXPERT_GROUPS 16

/* Each token's k experts and their weights.
 *   s = softmax(logits[t]) or sigmoid; value_e = s_e + bias_e (bias [E] fp32 or NULL: the
 *   choice's alone, as for balancing the experts' load).
 *   groups > 1: experts come in groups of E / groups (whole); a group's value is the sum of its
 *   group_best (1 or 2) best values, and only the top_groups best groups' experts are left.
 *   indices[t] = the k best values' experts, best first; weights[t][j] = scale s_e, divided by the
 *   chosen experts' sum with GBM_RENORMALIZE.
 * Equal values: the lower number first, for experts and groups alike. Values are compared as 64-bit
 * numbers (cut to 42 bits), the logits themselves where neither a bias nor group_best = 2 is involved.
 * Weights are formed in fp32 from the chosen logits: off by up to (2 D + 40) 2^-24 of themselves, D the largest distance of a
 * logit from the row's largest (softmax) or the largest logit's magnitude (sigmoid).
 * An expert whose logit or bias is -inf is never chosen: a slot that no expert is left for has index -1
 * and weight 0 (a padding token's logits are all -inf). A row with a NaN (softmax: or a logit of +inf; or a
 * NaN in the bias) has indices -1 and weights NaN.
 * k <= 32, k <= top_groups (E / groups); E <= 1024; groups <= 16, a divisor of E; scale finite: GBA_ERR_SHAPE.
 * Another score: GBA_ERR_ACT. logits: dtype, aligned to its size.
 *
 * offsets, rows (and slots): NULL, or the slots are sorted too, as moe_sort does. */
int moe_route(const void *logits, const float *bias, int32_t *indices, float *weights, int32_t *offsets, int32_t *rows,
              int32_t *slots, int64_t T, int64_t E, int64_t k, int64_t groups, int64_t top_groups, int group_best,
              int score, float scale, int dtype, int flags, void *workspace, size_t workspace_bytes);

/* dlogits [T,E] (`dtype`) from dweights [T,k]: the gradient of moe_route's weights for the chosen experts
 * (the choice itself has none, and neither has the bias). Experts that are not chosen get zeros, except
 * with softmax scores that are not renormalised. Slots of -1 add nothing. A token without any slot gets zeros, or
 * NaN where moe_route's weights are NaN for its logits (a NaN; softmax: or +inf), so that these do not pass for padding.
 * indices as moe_route leaves them (of an expert more than once in one row the terms add up, in the order of j). */
int moe_route_grad(const void *logits, const int32_t *indices, const float *dweights, void *dlogits, int64_t T, int64_t E,
                   int64_t k, int score, float scale, int dtype, int flags);

/* offsets [E+1] and rows [T,k] of indices [T,k], by a stable sort; slots [T k] or NULL: the slot t k + j of each
 * row, -1 for the rows from offsets[E] on. k may be more than E, as where one device holds some of a token's experts and the
 * others' slots are -1. workspace: moe_sort_workspace bytes, 16-byte aligned
 * (GBA_ERR_SCRATCH if less; contents neither needed nor kept). T = 0: offsets of zeros. */
int moe_sort(const int32_t *indices, int32_t *offsets, int32_t *rows, int32_t *slots, int64_t T, int64_t E, int64_t k,
             void *workspace, size_t workspace_bytes);

/* Bytes of workspace that sorting needs, 0 for few slots (or sizes that are refused); 256 KiB per 256 experts at most. */
size_t moe_sort_workspace(int64_t T, int64_t E, int64_t k);

/* --------------------------------------------------------- movement of rows -- */

/* out[rows[t][j]] = x[t]: x [T,H], out [R,H]. Rows of no slot are left as they were. */
int moe_dispatch(const void *x, const int32_t *rows, void *out, int64_t T, int64_t k, int64_t H, int64_t R, int dtype);

/* In the dtype of moe_combine and moe_combine_grad, beside the experts' rows' type: out and dout, the tokens' side,
 * are fp32, so that a loss is taken from sums that no 16-bit type has rounded, and its gradient is rounded once, in dy. */
enum { GBM_F32_TOKENS = 256 };

/* out[t] = sum over j of weights[t][j] y[rows[t][j]], in fp32, rounded once (not at all with GBM_F32_TOKENS):
 * y [R,H], out [T,H]. weights NULL: ones (the gradient of moe_dispatch). A slot of -1 adds weight times 0. */
int moe_combine(const void *y, const int32_t *rows, const float *weights, void *out, int64_t T, int64_t k, int64_t H,
                int64_t R, int dtype);

/* moe_combine's gradients: dy[rows[t][j]] = weights[t][j] dout[t] (rows of no slot are left as they were) and
 * dweights[t][j] = <dout[t], y[rows[t][j]]> in fp32 (0 for a slot of -1). Either may be NULL. */
int moe_combine_grad(const void *dout, const void *y, const int32_t *rows, const float *weights, void *dy, float *dweights,
                     int64_t T, int64_t k, int64_t H, int64_t R, int dtype);

/* ------------------------------------------------- 8-bit floats by blocks -- */

/* Values are OCP E4M3 codes (nearest, ties to even, largest 448) times an fp32 scale for each block:
 *   rows:     blocks of 128 along a row; codes [R,K], scales [ceil(K/128)][R].
 *   weights:  blocks of 128 x 128; codes [E,N,K], scales [E][ceil(N/128)][ceil(K/128)].
 * A block's scale is max |x| / 448, rounded to fp32, and its codes those nearest to 448 x / max (of
 * the exact quotient); a max under 448 2^-126 has the scale 2^-126 and codes nearest to x 2^126. With
 * GBM_POW2_SCALES the scale is the smallest power of two >= max / 448 (2^-126 at least). A block with an infinity or a
 * NaN has a scale of NaN and codes of zero. The last blocks of a row or column are shorter. K a multiple
 * of 16. */
enum { GBM_POW2_SCALES = 1 };

/* rows NULL: row t of X [T,K] to row t (k 1, R = T). Else to every row of rows [T,k], moe_dispatch in 8 bits:
 * codes and scales of rows of no slot are left as they were. */
int fp8_quantize(const void *X, const int32_t *rows, void *codes, float *scales, int64_t T, int64_t k, int64_t K, int64_t R,
                 int dtype, int flags);

/* X [R,K] = the values, rounded to `dtype`. */
int fp8_dequantize(const void *codes, const float *scales, void *X, int64_t R, int64_t K, int dtype);

/* codes, scales of W [E,N,K], and codes_t [E,K,N], scales_t [E][ceil(K/128)][ceil(N/128)] of each W_e
 * transposed (the same values; N a multiple of 16): what the forward product and the gradient of its input
 * take. Either pair may be NULL (both pointers), not both pairs. At most 4096 matrices, 2^30 blocks. */
int fp8_quantize_weights(const void *W, void *codes, float *scales, void *codes_t, float *scales_t, int64_t E, int64_t N,
                         int64_t K, int dtype, int flags);
int fp8_dequantize_weights(const void *codes, const float *scales, void *W, int64_t E, int64_t N, int64_t K, int dtype);

/* ---------------------------------------------------- products in 8 bits -- */

#define GBM_MAX_GROUPS 4096   /* experts of a product */

/* C = act(Z), Z = A.W^T + bias: A [M,K] in rows' form, W [N,K] in weights' form (E = 1); bias [N] or
 * NULL, C [M,N] and preact [M,N] or NULL (receives Z, rounded) in `dtype`. Each block's products are summed by the
 * matrix cores, multiplied by the two scales' product and added, in fp32: a scales' product below 2^-126 has fewer bits,
 * one of 2^128 or more is an infinity (blocks whose largest values' product is beyond 2^145). The matrix cores' own
 * rule, as measured: of each 8 consecutive products, those with less than 2^-13 of the largest's power of two lose what
 * is below that, towards zero. K a multiple of 16, at most 2^22; N of 8, at most 2^23; M at most 2^29. K = 0 gives
 * act(bias). workspace: NULL, or device memory (16-byte aligned) that lets calls with few output tiles split K
 * (deterministic; contents neither needed nor kept). */
int gemm_bias_act_fp8_block(const void *a_codes, const float *a_scales, const void *w_codes, const float *w_scales,
                            const void *bias, void *C, void *preact, int64_t M, int64_t N, int64_t K, int act, int dtype,
                            void *workspace, size_t workspace_bytes);

/* The same by expert: rows offsets[e] .. offsets[e+1] - 1 of A [T,K] times W_e, W [E,N,K], bias [E,N]. offsets
 * as in gba_experts.h (clamped to [0, T]; rows of no expert are neither read nor written). */
int grouped_gemm_bias_act_fp8_block(const void *a_codes, const float *a_scales, const int32_t *offsets, const void *w_codes,
                                    const float *w_scales, const void *bias, void *C, void *preact, int64_t T, int64_t E,
                                    int64_t N, int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes);

/* dA = (dC.W^T) * act'(z): the gradient of a product's input, through the activation that made that input
 * (A = act(z)). dC [M,K] in rows' form; W [N,K]: the forward weights transposed (codes_t, scales_t), so that N is the
 * forward product's depth and K its columns; z, dA [M,N]. act GBA_ACT_NONE: z may be NULL. act' as
 * grouped_gemm_act_grad's. Gradients of the weights are taken in 16 bits (grouped_gemm_wgrad). */
int gemm_act_grad_fp8_block(const void *dc_codes, const float *dc_scales, const void *w_codes, const float *w_scales,
                            const void *z, void *dA, int64_t M, int64_t N, int64_t K, int act, int dtype, void *workspace,
                            size_t workspace_bytes);
int grouped_gemm_act_grad_fp8_block(const void *dc_codes, const float *dc_scales, const int32_t *offsets, const void *w_codes,
                                    const float *w_scales, const void *z, void *dA, int64_t T, int64_t E, int64_t N, int64_t K,
                                    int act, int dtype, void *workspace, size_t workspace_bytes);

/* ---------------------------------------------------------- choice of kernel -- */

enum { GBM_RING = 0, GBM_PERSISTENT = 1, GBM_STREAM = 2 };
typedef struct {
    int32_t kind;             /* GBM_RING: tiles staged in LDS; GBM_PERSISTENT; GBM_STREAM: few rows, weights read once */
    int32_t tile_m, tile_n;   /* output tile of a workgroup */
    int32_t splits;           /* parts that K is split in (GBM_RING) */
} gbm_plan;

/* What a product in 8 bits of these sizes (T rows in all, K deep) takes on a device of `cus` compute units. Needs no
 * device. GBA_ERR_SHAPE and GBA_ERR_ALIGN as the products; T, N and K at least 1. */
int gbm_get_plan(int64_t T, int64_t E, int64_t N, int64_t K, size_t workspace_bytes, int cus, gbm_plan *plan);

#ifdef __cplusplus
}
#endif

#endif /* GBA_MOE_H */
