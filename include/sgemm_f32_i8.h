/*
 * sgemm_f32_i8 -- the norm that precedes a feed-forward block, and the block's
 * products with matrices in 8 bits, beside the gated block and the 4-bit weights of
 * sgemm_f32_ffn.h: the same library, types, conventions and return codes.
 *
 * Root-mean-square norm of M rows of K activations, after the residual R is added
 * where there is one:
 *
 *   H = X + R,  rstd[m] = 1 / sqrt(mean_k(H[m][k]^2) + eps),
 *   Y[m][k] = H[m][k] * rstd[m] * W[k]                      (sgemm_f32_rms_norm)
 *
 * and, given dY and the gradient dH that reaches H from behind the norm, its
 * backward pass is, with N = H * rstd,                      (sgemm_f32_rms_norm_bwd)
 *
 *   dX = dH + rstd * (dY * W - N * mean_k(dY * W * N)),  dW[k] = sum_m dY * N
 *
 * (dX is the gradient of X and of R alike).
 *
 * The 8-bit form holds a matrix as whole numbers q of -127..127 with one FP32
 * scale for each row, value = q * S[row]:
 *
 *   q = round(127 * x / max_k|x|),  S = max_k|x| / 127      (sgemm_f32_i8_quantize)
 *
 * halves to even; a row of zeros has S = 0 and q = 0, a row that holds an infinity or
 * NaN has S = NaN and q = 0. sgemm_f32_rms_norm_i8 gives Y in this form in
 * one pass: rstd is common to a row, so q = round(127 * H W / max|H W|) and S =
 * max|H W| * rstd / 127. The quotients are exact, but for FP32 rows of
 * sgemm_f32_rms_norm_i8, where one within 2^-44 of a half may round to either
 * side. With rows of X as tokens and rows of W as output features,
 *
 *   Y[m][f] = Sx[m] * Sw[f] * sum_k qx[m][k] * qw[f][k]     (sgemm_f32_i8)
 *   H = act(X Wg^T) * (X Wu^T), all three in 8 bits         (sgemm_f32_i8_glu)
 *
 * Sums of products are exact in 32 bits, so they do not depend on the order, nor a row's
 * results on the rows beside it: -128 is allowed as a stored number, and K is at most 131071
 * (SGEMM_F32_ERR_TOO_LARGE beyond). A sum is rounded to FP32 and multiplied by its two scales,
 * a rounding each; only the result has to lie in FP32's range, not what is between.
 *
 * Types. `dtype` is the type of every activation, norm weight, output and gradient
 * of a call: FP32, bfloat16 or IEEE half. Scales and rstd are FP32, and the stored numbers
 * int8. H is rounded to the type, and everything after it uses the rounded one, so that the
 * backward pass sees what the forward pass did. Sums over a row or over rows are held in FP32
 * (squares next to the ends of its range are summed times a power of two); each output is
 * rounded to the type once, from FP32. The backward pass forms dY W and dY W N in FP32, so these have
 * to lie in its range. A root mean square above 2^126 has an rstd below FP32's normal numbers, whose
 * rounding (2^-22 at most, relative, not 2^-24) is in what it scales.
 *
 * Infinities and NaN stay in their rows (dW: in their columns): a row of H that holds an infinity has
 * rstd = 0, and Y = 0 but for the infinity, where it is NaN; one that holds NaN is NaN. With eps = 0 a row
 * of zeros has rstd = inf and Y = NaN, and one whose root mean square is below 2^-128 rstd = inf. A scale that is infinite or NaN gives what the product of FP32
 * numbers gives.
 *
 * Layout. Matrices are row-major with unit column stride and a leading
 * dimension in elements, any base aligned to its element serves; W of the norm,
 * dW, scales and rstd are vectors of unit stride. Outputs must not overlap inputs or each
 * other, but for these, element for element (the same base and leading
 * dimension): H may be X or R; Y may be X or R, where H is not; dX may be dH
 * or dY. Padding between rows is neither read nor written.
 *
 * Ownership, asynchrony, determinism (no atomics; a fixed summation order for a
 * device and a call's shape) and thread safety are those of sgemm_f32.h. A
 * call only enqueues kernels, so it can be captured in a graph. Calls that may run at
 * the same time need workspaces of their own. Work runs on the current
 * device, which has to own the stream and the memory.
 *
 * Empty sums are zero: K == 0 gives Y = 0 for the products (scales are then not read), S = 0,
 * and rstd = 1 / sqrt(eps); M == 0 gives dW = 0. A call whose outputs are empty touches no memory.
 *
 * Return codes: those of sgemm_f32.h, each argument under one number in every
 * entry point (the first bad one is reported, in this order):
 *   -17 dtype   -18 act    -1 M < 0   -2 F < 0   -3 K < 0
 *   -40 eps is negative, infinite or NaN
 *   -5 X        -6 ldx     -44 Sx     -38 R      -39 ldr
 *   -45 dY      -46 lddy
 *   -7 W (Wg, Q; rms_norm_i8 has both, W first)  -8 ldw (ldwg, ldq)    -32 S (Sw, Sg)
 *   -19 Wu      -20 ldwu   -36 Su
 *   -41 H (the norm's)     -42 ldh    -43 rstd
 *   -23 dH      -24 lddh
 *   -10 Y (H of i8_glu, X of i8_dequantize)      -11 ldy (ldh, ldx)
 *   -25 dX      -26 lddx   -27 dW
 *   -16 workspace NULL with a nonzero size or not 16-byte aligned
 *   -12 output pointer NULL
 *   SGEMM_F32_ERR_TOO_LARGE   a size exceeds what the kernels can index
 *   SGEMM_F32_ERR_WORKSPACE   workspace_bytes below what the _ws_size reports
 * A pointer is checked (not NULL, aligned to its element) where it is read or
 * written; leading dimensions of operands that are not NULL always.
 */
#ifndef SGEMM_F32_I8_H
#define SGEMM_F32_I8_H

#include <stdint.h>

#include "sgemm_f32_ffn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Y = rms_norm(X + R) * W. X, R, H, Y: M x K; W: K. R may be NULL (H = X).
 * H and rstd (M values), where not NULL, receive what sgemm_f32_rms_norm_bwd needs;
 * H is also the residual stream's next value. */
SGEMM_F32_API int sgemm_f32_rms_norm(int dtype, int64_t M, int64_t K, float eps, const void *X,
                                     int64_t ldx, const void *R, int64_t ldr, const void *W, void *H,
                                     int64_t ldh, float *rstd, void *Y, int64_t ldy, void *stream);

/* The same with Y in 8 bits: Q (M x K), S (M values). */
SGEMM_F32_API int sgemm_f32_rms_norm_i8(int dtype, int64_t M, int64_t K, float eps, const void *X,
                                        int64_t ldx, const void *R, int64_t ldr, const void *W, void *H,
                                        int64_t ldh, int8_t *Q, int64_t ldq, float *S, void *stream);

/* The gradients of sgemm_f32_rms_norm for dY (M x K), from H, W and rstd. dH
 * (M x K), the gradient that reaches H from behind, may be NULL (none). dX (M x K) and
 * dW (K) are overwritten; each may be NULL, and is then not computed. The
 * workspace holds partial sums of dW (sgemm_f32_rms_norm_bwd_ws_size); without
 * dW none is needed. */
SGEMM_F32_API int sgemm_f32_rms_norm_bwd(int dtype, int64_t M, int64_t K, const void *dY, int64_t lddy,
                                         const void *W, const void *H, int64_t ldh, const float *rstd,
                                         const void *dH, int64_t lddh, void *dX, int64_t lddx, void *dW,
                                         void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of sgemm_f32_rms_norm_bwd (host only). Returns 0, -17, -1,
 * -3, -12 or SGEMM_F32_ERR_TOO_LARGE. */
SGEMM_F32_API int sgemm_f32_rms_norm_bwd_ws_size(int dtype, int64_t M, int64_t K, size_t *bytes);

/* X (M x K) to 8 bits: Q (M x K), S (M values). */
SGEMM_F32_API int sgemm_f32_i8_quantize(int dtype, int64_t M, int64_t K, const void *X, int64_t ldx,
                                        int8_t *Q, int64_t ldq, float *S, void *stream);

/* X[m][k] = q * S[m], rounded to FP32 and then to the type. */
SGEMM_F32_API int sgemm_f32_i8_dequantize(int dtype, int64_t M, int64_t K, const int8_t *Q, int64_t ldq,
                                          const float *S, void *X, int64_t ldx, void *stream);

/* Y = X W^T of matrices in 8 bits, Y in `dtype`. X: M x K, W: F x K, Y: M x F. */
SGEMM_F32_API int sgemm_f32_i8(int dtype, int64_t M, int64_t F, int64_t K, const int8_t *X, int64_t ldx,
                               const float *Sx, const int8_t *W, int64_t ldw, const float *Sw, void *Y,
                               int64_t ldy, void *stream);

/* H = act(X Wg^T) * (X Wu^T) of matrices in 8 bits, H in `dtype`. */
SGEMM_F32_API int sgemm_f32_i8_glu(int dtype, int act, int64_t M, int64_t F, int64_t K, const int8_t *X,
                                   int64_t ldx, const float *Sx, const int8_t *Wg, int64_t ldwg,
                                   const float *Sg, const int8_t *Wu, int64_t ldwu, const float *Su,
                                   void *H, int64_t ldh, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_F32_I8_H */
