/*
 * sgemm_f32_ffn -- the gated feed-forward block and its 4-bit form, beside the
 * products of sgemm_f32.h: the same library, conventions and return codes.
 *
 * The block multiplies M rows of K activations by two weight matrices of F
 * output features and gates one product with the other:
 *
 *   G = X Wg^T,  U = X Wu^T,  H = act(G) * U                (sgemm_f32_glu)
 *
 * and, given dH, its backward pass is                       (sgemm_f32_glu_bwd)
 *
 *   dU = dH * act(G),  dG = dH * U * act'(G),
 *   dX = dG Wg + dU Wu,  dWg = dG^T X,  dWu = dU^T X.
 *
 * The 4-bit form holds a weight as a whole number q of 0..15 with a scale
 * (and a zero point) shared by `group` consecutive inputs of one output:
 *
 *   W[n][k] = (q[n][k] - zero[n][k / group]) * scale[n][k / group],
 *
 * zero = 8 where no zero points are given. sgemm_f32_w4_quantize makes it,
 * sgemm_f32_w4_dequantize expands it, sgemm_f32_w4 multiplies by it
 * (Y = X W^T) and sgemm_f32_w4_glu gates two such products.
 *
 * Types. `dtype` is the type of every activation, weight, scale, zero point,
 * output and gradient of a call: FP32, bfloat16 or IEEE half. Products are
 * exact and sums are held in FP32 whatever the type; outputs are rounded
 * once. Where a 16-bit call has to keep a value between two products (dG and
 * dU, which the matrix cores read in the type), it is rounded once more, or,
 * where M * F <= 16384, kept in two parts. In half, which spans less than the
 * gradients do, they are kept times a power of two, one for all of a call's,
 * that brings the largest finite one to the top of the type's range: each is
 * then off by half a step, or by 2^-40 of that largest one where this is more,
 * and none overflows. G and U are kept for the backward
 * pass in FP32 (`P`), so that no rounding comes before the derivative.
 *
 * Infinities and NaN stay in the rows and columns whose sums they enter. Where dG
 * and dU are kept in two parts, an infinity in X or a weight gives NaN there. With
 * 4-bit weights an infinity in X, or values of a row whose magnitudes sum to more
 * than 2^122, may give NaN or an infinity where the exact sum is finite (the numbers
 * are summed before their zero point is taken off), and parts of FP32 values below 2^-126 count as
 * zero.
 *
 * Layout. Every matrix is row-major with unit column stride and a leading
 * dimension in elements (element (r, c) at base[r * ld + c]); a weight has one
 * row of K inputs for each output feature. Any leading dimension and any base
 * aligned to its element serves; rows that are whole 16-byte chunks are
 * fastest. Q holds two weights a byte, the even k in the low half, in rows of
 * ldq >= (K + 1) / 2 bytes; the unused half of an odd K's last byte is written
 * as zero and ignored on reading. Scales and zero points are F x G matrices,
 * G = ceil(K / group).
 *
 * Outputs must not overlap inputs or each other. Padding between rows is
 * neither read nor written. Ownership, asynchrony, determinism (no atomics;
 * a fixed summation order for a device and a call's shape) and thread safety
 * are those of sgemm_f32.h, and a call only enqueues kernels, so it can be
 * captured in a graph. Calls that may run at the same time need workspaces
 * of their own. Work runs on the current device, which has to own the stream
 * and the memory.
 *
 * Empty sums are zero: K == 0 gives H = 0 and Y = 0; M == 0 gives dWg = dWu =
 * 0; F == 0 gives dX = 0. A call whose outputs are empty touches no memory.
 *
 * Return codes: those of sgemm_f32.h, each argument under one number in every
 * entry point (the first bad one is reported, in this order):
 *   -17 dtype   -18 act    -1 M < 0   -2 F < 0   -3 K < 0   -31 group
 *   -5 X (or W, the matrix to quantise)          -6 ldx (ldw)
 *   -7 Wg (or Q, Qg)       -8 ldwg (ldq)         -19 Wu (Qu)   -20 ldwu
 *   -32 scales (Sg)        -33 lds               -36 Su
 *   -34 zero points (Zg)   -35 ldz               -37 Zu
 *   -21 P       -22 ldp    -23 dH     -24 lddh
 *   -10 H (Y, or W the expanded matrix)          -11 ldh (ldy, ldw)
 *   -25 dX      -26 lddx   -27 dWg    -28 lddwg  -29 dWu      -30 lddwu
 *   -16 workspace NULL with a nonzero size or not 16-byte aligned
 *   -12 output pointer NULL
 *   SGEMM_F32_ERR_WORKSPACE   workspace_bytes below what the _ws_size reports
 *   SGEMM_F32_ERR_TOO_LARGE   a size exceeds what the kernels can index
 * A pointer is checked (not NULL, aligned to its element) where it is read or
 * written; leading dimensions always.
 */
#ifndef SGEMM_F32_FFN_H
#define SGEMM_F32_FFN_H

#include "sgemm_f32.h"

#ifdef __cplusplus
extern "C" {
#endif

enum sgemm_f32_dtype {
    SGEMM_F32_DTYPE_F32 = 0,
    SGEMM_F32_DTYPE_BF16 = 1,
    SGEMM_F32_DTYPE_F16 = 2
};

/* The gate's activation. */
enum sgemm_f32_act {
    SGEMM_F32_ACT_SILU = 0,      /* g / (1 + exp(-g)) */
    SGEMM_F32_ACT_GELU = 1,      /* g * (1 + erf(g / sqrt(2))) / 2 */
    SGEMM_F32_ACT_GELU_TANH = 2, /* g * (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 */
    SGEMM_F32_ACT_RELU = 3       /* max(g, 0); slope 0 at 0 */
};

/* H = act(X Wg^T) * (X Wu^T). X: M x K, Wg and Wu: F x K, H: M x F. P, when
 * not NULL, receives what sgemm_f32_glu_bwd needs: an FP32 matrix of M rows,
 * G in columns 0 .. F-1 and U in columns F .. 2F-1 (ldp >= 2F). */
SGEMM_F32_API int sgemm_f32_glu(int dtype, int act, int64_t M, int64_t F, int64_t K, const void *X,
                                int64_t ldx, const void *Wg, int64_t ldwg, const void *Wu,
                                int64_t ldwu, void *H, int64_t ldh, float *P, int64_t ldp,
                                void *stream);

/* The gradients of sgemm_f32_glu for dH (M x F), from its inputs and P. dX
 * (M x K), dWg and dWu (F x K) are overwritten; each may be NULL, and is then
 * not computed (its leading dimension is ignored). The workspace holds dG and
 * dU (sgemm_f32_glu_bwd_ws_size). */
SGEMM_F32_API int sgemm_f32_glu_bwd(int dtype, int act, int64_t M, int64_t F, int64_t K,
                                    const void *X, int64_t ldx, const void *Wg, int64_t ldwg,
                                    const void *Wu, int64_t ldwu, const float *P, int64_t ldp,
                                    const void *dH, int64_t lddh, void *dX, int64_t lddx,
                                    void *dWg, int64_t lddwg, void *dWu, int64_t lddwu,
                                    void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of sgemm_f32_glu_bwd on a device with num_cus compute
 * units (host only). Returns 0, -17, -1, -2, -3, -12 or
 * SGEMM_F32_ERR_TOO_LARGE. */
SGEMM_F32_API int sgemm_f32_glu_bwd_ws_size(int dtype, int64_t M, int64_t F, int64_t K,
                                            int num_cus, size_t *bytes);

/* W (F x K) to 4 bits. `group` is a positive multiple of 32, or any value of
 * at least K (one group a row). With Z NULL the form is symmetric: scale =
 * max|w| / 7, q = round(w / scale) + 8. With Z: lo = min(w, 0), hi = max(w, 0),
 * scale = (hi - lo) / 15, zero = round(-lo / scale), q = round(w / scale) + zero,
 * all within 0..15. The scale is rounded to the type first and quotients by
 * the rounded one are taken exactly; halves round to even. A scale of 0 gives q =
 * zero (8, or 0 with Z). A group that holds an infinity or NaN gets the scale
 * NaN. */
SGEMM_F32_API int sgemm_f32_w4_quantize(int dtype, int64_t F, int64_t K, int64_t group,
                                        const void *W, int64_t ldw, void *Q, int64_t ldq, void *S,
                                        int64_t lds, void *Z, int64_t ldz, void *stream);

/* W[n][k] = (q - zero) * scale, rounded once where q - zero is exact in FP32 (as
 * with whole zero points, which sgemm_f32_w4_quantize makes), and otherwise
 * once more. Z NULL: zero = 8. */
SGEMM_F32_API int sgemm_f32_w4_dequantize(int dtype, int64_t F, int64_t K, int64_t group,
                                          const void *Q, int64_t ldq, const void *S, int64_t lds,
                                          const void *Z, int64_t ldz, void *W, int64_t ldw,
                                          void *stream);

/* Y = X W^T with W in 4 bits. X: M x K, W: F x K, Y: M x F. */
SGEMM_F32_API int sgemm_f32_w4(int dtype, int64_t M, int64_t F, int64_t K, int64_t group,
                               const void *X, int64_t ldx, const void *Q, int64_t ldq,
                               const void *S, int64_t lds, const void *Z, int64_t ldz, void *Y,
                               int64_t ldy, void *stream);

/* H = act(X Wg^T) * (X Wu^T) with both weights in 4 bits, in matrices of the
 * same leading dimensions; Zg and Zu are both given or both NULL (-37). */
SGEMM_F32_API int sgemm_f32_w4_glu(int dtype, int act, int64_t M, int64_t F, int64_t K,
                                   int64_t group, const void *X, int64_t ldx, const void *Qg,
                                   const void *Qu, int64_t ldq, const void *Sg, const void *Su,
                                   int64_t lds, const void *Zg, const void *Zu, int64_t ldz,
                                   void *H, int64_t ldh, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F32_FFN_H */
