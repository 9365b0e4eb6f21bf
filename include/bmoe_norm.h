/*
 * bmoe_norm.h - layer norm in front of a ButterflyMoE layer (bmoe.h), forward
 * and backward.
 *
 * The pages put their expert layers in the place of a transformer block's
 * feed-forward part (ButterflyMoE, gist.science/nl/paper/2601.13563, §2;
 * ButterflyViT, gist.science/pt/paper/2603.06746, §2); a block of that kind
 * feeds the layer the norm of its residual stream.  For every row
 *     s    = x + residual                       (s = x without a residual)
 *     mean = sum_j s_j / width,   var = sum_j (s_j - mean)^2 / width
 *     rstd = 1 / sqrt(var + eps)
 *     y_j  = (s_j - mean) rstd gamma_j + beta_j.
 * s is rounded to the activation dtype first and the norm is that of the
 * rounded row, so the backward, which reads the stored s, sees the forward's
 * values.  Sums run in fp32 over a row held in registers: the mean's rounding
 * is taken from the sum of the centred values and given back to the mean, the
 * variance and y, so a row far from 0 is normed as well as one around it and a
 * constant row gives y = beta.  Squares that leave fp32, or vanish in it beside
 * an eps below 2^-100, are summed at another scale: a finite row is normed
 * whatever its size (entries up to 2^127; rstd is infinite for deviations below
 * 2^-128).
 *
 * Widths 1 .. 16384, rows 0 .. 2^24; arrays are row-major and
 * dense, aligned to their element size (16-byte alignment and a width that is
 * a multiple of 8 are fastest).  Memory rules as in bmoe.h: every
 * pointer is caller-owned device memory, nothing is allocated or
 * synchronised, all work is enqueued on `stream`, results do not depend on
 * scheduling, and all errors but BMOE_ERR_HIP are found before anything is
 * enqueued.
 */
#ifndef BMOE_NORM_H
#define BMOE_NORM_H

#include "bmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Forward.
 *   x         [rows][width] of dtype (bmoe_dtype), read only.
 *   residual  [rows][width] of dtype or NULL, read only.
 *   gamma     [width] fp32 or NULL (all ones);  beta [width] fp32 or NULL
 *             (all zeros), read only.
 *   eps       finite, not negative.
 *   sum       [rows][width] of dtype, written with s: given exactly when
 *             residual is; may be the same buffer as x or residual.
 *   y         [rows][width] of dtype, written; may be the same buffer as x or
 *             residual (not as sum).  Without a residual x is the row that the
 *             backward reads: over it y serves a forward alone.
 *   mean, rstd  [rows] fp32, written, for the backward: both or neither NULL.
 * A row that holds a NaN or an infinity becomes NaN, other rows are not
 * affected.  Errors: BMOE_ERR_SHAPE (rows, width, eps), BMOE_ERR_DTYPE,
 * BMOE_ERR_NULL (also sum without residual, mean without rstd and the other
 * way round), BMOE_ERR_ALIGN, BMOE_ERR_ALIAS, BMOE_ERR_DEVICE, BMOE_ERR_HIP. */
bmoe_status bmoe_layer_norm_forward(int32_t rows, int32_t width, int32_t dtype, const void* x, const void* residual,
                                    const float* gamma, const float* beta, float eps, void* sum, void* y, float* mean,
                                    float* rstd, hipStream_t stream);

/* Device workspace bytes of bmoe_layer_norm_backward (per-workgroup partial
 * sums of the weights' gradients; 0 for few rows, whose gradients need none). */
bmoe_status bmoe_layer_norm_backward_workspace(int32_t rows, int32_t width, size_t* bytes);

/* Backward at the forward's s, mean and rstd.  With xhat = (s - mean) rstd and
 * v = gamma dy, per row
 *     dx = rstd (v - sum_j v_j / width - xhat sum_j v_j xhat_j / width) + d_sum
 * (the same gradient goes to x and to the residual), and over all rows
 *     dgamma = sum dy xhat,   dbeta = sum dy.
 *   dy        [rows][width] of dy_dtype: fp32 (the input gradient of
 *             bmoe_layer_backward) or dtype, read only.
 *   s         [rows][width] of dtype: the forward's sum (x without a
 *             residual), read only.
 *   gamma     [width] fp32 or NULL, read only;  mean, rstd [rows] fp32, read
 *             only.
 *   d_sum     [rows][width] of dtype or NULL: gradient that reaches s past the
 *             norm (the residual stream's own), read only.
 *   dx        [rows][width] of dtype, written; may be the same buffer as s or
 *             d_sum, or as dy when dy_dtype is dtype.
 *   dgamma, dbeta  [width] fp32, written (zero for rows = 0): both or neither
 *             NULL.
 *   workspace at least bmoe_layer_norm_backward_workspace bytes, 16-byte
 *             aligned, contents undefined after; may be NULL when dgamma is, or when
 *             that is 0.
 * Column sums are fp32, added in an order that the sizes and the alignment
 * alone decide.  Errors as above, and BMOE_ERR_WORKSPACE. */
bmoe_status bmoe_layer_norm_backward(int32_t rows, int32_t width, int32_t dtype, int32_t dy_dtype, const void* dy,
                                     const void* s, const float* gamma, const float* mean, const float* rstd,
                                     const void* d_sum, void* dx, float* dgamma, float* dbeta, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BMOE_NORM_H */
