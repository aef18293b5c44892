/*
 * gba_experts.h -- C ABI of libgba_experts: products grouped by expert, forward
 * and backward, and microscaled 4-bit floating point (quantisation and product),
 * for MI355X (gfx950). It sits beside libgba (gba.h) and shares its enums
 * (gba_dtype, gba_act) and status codes.
 *
 * Conventions shared by every entry point (as gba.h unless stated):
 *   - All array arguments are DEVICE pointers owned by the caller, dense and
 *     row-major. The library allocates nothing and keeps no pointer after a call.
 *   - Pointers must be 16-byte aligned (offsets: 4-byte); row lengths must be
 *     multiples of 8 values in 16 bits, of 32 values in 4 bits: GBA_ERR_ALIGN.
 *   - A product has at most 2^29 rows (T; M of the dense 4-bit product), an
 *     operand to be quantised less than 2^31: GBA_ERR_SHAPE.
 *   - Accumulation is fp32; each output is rounded once, to nearest even.
 *     Activations are gba.h's (GELU within 8e-6 of |z| Phi(-|z|)). Their
 *     derivatives are within 4e-7; below z = -1.5 within (A + 8) 2^-23 of
 *     themselves, A the argument of their exponential (z^2/2 for GELU).
 *   - Argument errors are reported synchronously, before any launch. Work is
 *     enqueued on the calling thread's stream (gbx_set_stream) and runs
 *     asynchronously. Nothing synchronises, allocates or copies, so every entry
 *     point can be recorded in a HIP graph.
 *   - No output may overlap an input or another output: GBA_ERR_ALIAS.
 *   - Unknown flag bits: GBA_ERR_SHAPE.
 *   - A launch failure returns GBA_ERR_HIP (gbx_last_hip_error() gives the
 *     code); a device that is not gfx950 GBA_ERR_DEVICE.
 *
 * Groups. T rows are sorted by expert: expert e owns rows offsets[e] ..
 * offsets[e+1] - 1, with offsets an array of E + 1 int32 in device memory (the
 * host never reads it, so a router's result is used without a synchronisation).
 * Experts may be empty, E >= 1. Each offset is taken clamped to [0, T], and an
 * expert whose end lies before its start as empty, so that no value of offsets
 * leads outside the arrays. Rows that belong to no expert (before offsets[0],
 * from offsets[E] on) are neither read nor written. Offsets that decrease are
 * the caller's error: which rows are then written is not defined.
 */
#ifndef GBA_EXPERTS_H
#define GBA_EXPERTS_H

#include "gba.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Stream for this thread's later calls of this library (a hipStream_t). */
int gbx_set_stream(void *hip_stream);
int gbx_last_hip_error(void);
const char *gbx_version(void);

/* Most experts in one call. */
#define GBX_MAX_EXPERTS 4096

/* C[r] = act(Z[r]), Z[r] = A[r].W_e + bias_e for the rows r of each expert e.
 * A: [T,K]; W: [E,K,N], or [E,N,K] with GBA_TRANSPOSE_B in flags; bias: [E,N] or
 * NULL; C: [T,N]; preact: [T,N] or NULL, receives Z rounded (what
 * grouped_gemm_act_grad takes as z). All `dtype` (gba_dtype). K == 0 gives
 * act(bias_e). workspace: NULL, or device memory that lets calls with few
 * output tiles split K (deterministic; contents neither needed nor kept).
 * Sizes: N <= 2^23, K <= 2^21, else GBA_ERR_SHAPE. */
int grouped_gemm_bias_act(const void *A, const int32_t *offsets, const void *W, const void *bias,
                          void *C, void *preact, int64_t T, int64_t E, int64_t N, int64_t K,
                          int act, int dtype, int flags, void *workspace, size_t workspace_bytes);

/* dA[r] = (dC[r].W_e^T) * act'(z[r]): the gradient of the product's input,
 * carried through the activation that made that input (A = act(z)).
 * dC: [T,N]; W and flags as in the forward call ([E,K,N], or [E,N,K] with
 * GBA_TRANSPOSE_B); z, dA: [T,K]. act GBA_ACT_NONE: dA = dC.W_e^T and z may be
 * NULL. relu'(0) is 0; at z = +-inf every derivative is its limit; NaN gives NaN.
 * Sizes: N <= 2^21 (the depth of this product), K <= 2^23, else GBA_ERR_SHAPE. */
int grouped_gemm_act_grad(const void *dC, const int32_t *offsets, const void *W, const void *z,
                          void *dA, int64_t T, int64_t E, int64_t N, int64_t K, int act, int dtype,
                          int flags, void *workspace, size_t workspace_bytes);

/* grouped_gemm_wgrad flags beside GBA_TRANSPOSE_B. */
enum {
    GBX_OUT_F32 = 16,   /* dW and dbias are fp32 */
    GBX_ACCUMULATE = 32 /* add to dW and dbias (needs GBX_OUT_F32) */
};

/* dW_e = A_e^T.dC_e, stored [E,K,N], or dC_e^T.A_e, stored [E,N,K] with
 * GBA_TRANSPOSE_B (the layout W has in the forward call); dbias_e = the sum of
 * dC's rows of e (dbias [E,N], or NULL: not computed). A: [T,K], dC: [T,N].
 * An empty expert's gradients are written as zeros (left as they are with
 * GBX_ACCUMULATE). dW and dbias have `dtype`, or are fp32 with GBX_OUT_F32.
 * T == 0: zeros. K and N at most 2^23. */
int grouped_gemm_wgrad(const void *A, const void *dC, const int32_t *offsets, void *dW,
                       void *dbias, int64_t T, int64_t E, int64_t N, int64_t K, int dtype,
                       int flags, void *workspace, size_t workspace_bytes);

/* Microscaled 4-bit floating point (OCP MX, MXFP4): blocks of 32 values along a
 * row share a scale 2^(s - 127), s an 8-bit exponent (E8M0; 255 is NaN); each
 * value is a 4-bit E2M1 code (sign, then 0 .5 1 1.5 2 3 4 6).
 *   codes:  [M][K/2] bytes, code 2i in the low half of byte i.
 *   scales: [ceil(K/128)][M][4] bytes: block b of row m is byte b%4 of entry
 *           [b/4][m]; the bytes of blocks past K are written as 0, and a product
 *           needs them to be no NaN (255). One plane feeds one matrix
 *           instruction step of 128 values. */

/* Quantise X [M,K] (`dtype`): s = floor(log2(max |x|)) - 2 + 127 over the block,
 * at least 0; codes nearest to x / 2^(s-127), ties to the even code, magnitudes
 * over 6 to 6. A block of zeros has s = 0 and codes of zero (the sign kept). A
 * block with an infinity or a NaN has s = 255 and codes of zero. */
int mx4_quantize(const void *X, void *codes, void *scales, int64_t M, int64_t K, int dtype);

/* X [M,K] = the values, rounded to `dtype` (exact in bf16; in fp16 where its
 * range allows, else infinity or rounded subnormals). */
int mx4_dequantize(const void *codes, const void *scales, void *X, int64_t M, int64_t K,
                   int dtype);

/* C = act(A.W^T + bias): A [M,K] and W [N,K] in 4 bits (codes and scales as
 * above), bias [N] or NULL and C [M,N] in `dtype`. K a multiple of 32, at most
 * 2^23; N a multiple of 8. workspace as grouped_gemm_bias_act. */
int gemm_bias_act_mx4(const void *a_codes, const void *a_scales, const void *w_codes,
                      const void *w_scales, const void *bias, void *C, int64_t M, int64_t N,
                      int64_t K, int act, int dtype, void *workspace, size_t workspace_bytes);

/* The same by expert: A [T,K] sorted by expert, w_codes [E][N][K/2], w_scales
 * the planes of the [E*N, K] matrix ([ceil(K/128)][E*N][4]), bias [E,N]. */
int grouped_gemm_bias_act_mx4(const void *a_codes, const void *a_scales, const int32_t *offsets,
                              const void *w_codes, const void *w_scales, const void *bias, void *C,
                              int64_t T, int64_t E, int64_t N, int64_t K, int act, int dtype,
                              void *workspace, size_t workspace_bytes);

/* What a call of these sizes runs on a device of `cus` compute units: the output
 * tile of a workgroup, whether the persistent kernel walks such tiles, the K
 * ranges whose partial sums a second pass joins (1: none), and whether the
 * weights are read non-temporally. workspace_bytes: of a workspace that the call is given (0:
 * none). T is M for the dense 4-bit product. Launches nothing and needs no device. Sizes as
 * in the call: GBA_ERR_SHAPE, GBA_ERR_ALIGN; also GBA_ERR_SHAPE for another op, sizes of 0 or cus < 1. */
enum {
    GBX_FORWARD = 0,    /* grouped_gemm_bias_act */
    GBX_ACT_GRAD = 1,   /* grouped_gemm_act_grad */
    GBX_WGRAD = 2,      /* grouped_gemm_wgrad */
    GBX_WGRAD_BIAS = 3, /* the same with dbias */
    GBX_MX4 = 4         /* gemm_bias_act_mx4 (E = 1), grouped_gemm_bias_act_mx4 */
};
typedef struct {
    int32_t tile_m, tile_n;
    int32_t persistent;
    int32_t splits;
    int32_t non_temporal;
} gbx_plan;
int gbx_get_plan(int op, int64_t T, int64_t E, int64_t N, int64_t K, size_t workspace_bytes,
                 int cus, gbx_plan *plan);

#ifdef __cplusplus
}
#endif

#endif /* GBA_EXPERTS_H */
