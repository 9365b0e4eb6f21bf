/*
 * bmoe_update.h - from the gradient of a latent substrate to the next packed
 * substrate: the orthogonalised update and the latent weights' step.
 *
 * bmoe_layer_backward (bmoe_train.h) leaves dL/dW of every latent substrate.
 * The pages train the latent weights through a ternary quantiser and a
 * straight-through estimator (gist.science/nl/paper/2601.13563, §2 "Drie
 * Fasen van de Methode"; gist.science/zh/paper/2601.13563, technical summary
 * §2.2) and name neither the optimiser nor the quantiser's threshold; the
 * choices here are this library's: an update with orthonormalised rows (or
 * columns), and the mean-magnitude quantiser.
 *
 * Memory rules as in bmoe.h: every pointer is caller-owned device memory,
 * nothing is allocated or synchronised, all work is enqueued on `stream`,
 * results do not depend on scheduling, and all errors but BMOE_ERR_HIP are
 * found before anything is enqueued.  Calls that may overlap in time need
 * workspaces and outputs of their own.
 */
#ifndef BMOE_UPDATE_H
#define BMOE_UPDATE_H

#include "bmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Momentum step and orthogonalisation of a matrix gradient G [rows][cols]:
 *     M' = mu M + G
 *     U  = G + mu M' (nesterov 1),  M' (nesterov 0),  G (without momentum)
 *     X  = U / ||U||_F            (X = 0 for U = 0)
 *     five times  X <- a X + (b A + c A A) X,  A = X X^T  (on the smaller side)
 *     with (a, b, c) = (3.4445, -4.7750, 2.0315):
 * every singular value of U ends between 0.68 and 1.21 unless it was smaller
 * than 1.5e-3 of ||U||_F (1e-3 of it ends at 0.47), its singular vectors stay.
 * O = X.
 *
 * Precision.  Products run on the matrix cores in fp16 with fp32 sums, every
 * factor scaled by a power of two to the middle of fp16's range; X is kept as
 * fp16 and an 8-bit second term where a rounding of it would grow most, and the
 * symmetric factors' diagonals are corrected in fp32.  Measured
 * ||O - O_exact|| / ||O_exact|| before O's rounding to bf16 (1.7e-3 by itself):
 * below 1e-3 for gradients of full rank whose singular values fall off like
 * 1 / k or slower, 3.5e-3 at rank min(rows, cols) / 8, 6e-3 to 8e-3 at rank one,
 * for sides of 48 to 16384.  Gradients of both types take this one path; there
 * is none in fp32.  M' is fp32.  A NaN or an infinity in U makes all of O NaN.
 *
 * rows, cols in [1, 16384].
 *   grad      [rows][cols] of grad_dtype (bmoe_dtype), read only.
 *   momentum  [rows][cols] fp32 or NULL, read only;  momentum_out [rows][cols]
 *             fp32, written with M' (given exactly when momentum is; may be
 *             the same buffer as momentum).
 *   mu        in [0, 1];  nesterov 0 or 1 (both unused without momentum).
 *   out       [rows][cols] bf16, written.
 *   workspace at least bmoe_orthogonalize_workspace bytes, 256-byte aligned,
 *             contents undefined after.
 * Arrays aligned to their element size.  Errors: BMOE_ERR_SHAPE,
 * BMOE_ERR_DTYPE, BMOE_ERR_NULL, BMOE_ERR_ALIGN, BMOE_ERR_ALIAS (an output or
 * the workspace overlaps another array), BMOE_ERR_WORKSPACE,
 * BMOE_ERR_DEVICE, BMOE_ERR_HIP. */
bmoe_status bmoe_orthogonalize_workspace(int32_t rows, int32_t cols, size_t* bytes);
bmoe_status bmoe_orthogonalize(int32_t rows, int32_t cols, int32_t grad_dtype, const void* grad, const float* momentum,
                               float* momentum_out, float mu, int32_t nesterov, void* out, void* workspace,
                               size_t workspace_bytes, hipStream_t stream);

/* Step of a latent substrate W [rows][cols] and its ternary codes:
 *     W'    = fl32((1 - decay) W - step O)      (W' = W without O)
 *     scale = sum |W'| / (rows cols)
 *     code  = sign(W') where 2 |W'| > scale, else 0
 * (the nearest of -1, 0, 1 to W' / scale, a tie to 0).  W' is computed in fp64
 * and rounded once, the sum and the comparison are fp64: the codes do not
 * depend on an order of summation.  A NaN weight gets code 0; a sum that is
 * NaN or infinite makes every code 0.
 *   w        [rows][cols] fp32 (16-byte aligned), read only.
 *   o        [rows][cols] bf16 (16-byte aligned) or NULL, read only.
 *   w_out    [rows][cols] fp32 (16-byte aligned), written with W'; given
 *            exactly when o is; may be the same buffer as w.
 *   packed   [rows][cols / 16] words (16-byte aligned), written in
 *            bmoe_pack_ternary's format: w_base of bmoe_layer.
 *   scale    1 fp32, written, or NULL: the w_scale under which the codes
 *            stand for W'.  bmoe_layer's w_scale is a host value that this call
 *            does not touch: a caller whose layer computes with scale * codes
 *            copies scale back and sets it, one whose layer keeps a fixed w_scale
 *            (its output then does not depend on |W'|) leaves it.
 *   workspace at least bmoe_substrate_step_workspace bytes, 16-byte aligned,
 *            contents undefined after; may be NULL when that is 0 (few
 *             weights).
 * rows >= 1, cols a positive multiple of 16, rows * cols below 2^31; step and
 * decay finite.  A layer's prepared buffer (bmoe_prepare) is stale after its
 * w_base changed.  Errors: BMOE_ERR_SHAPE, BMOE_ERR_NULL, BMOE_ERR_ALIGN,
 * BMOE_ERR_ALIAS, BMOE_ERR_WORKSPACE, BMOE_ERR_DEVICE, BMOE_ERR_HIP. */
bmoe_status bmoe_substrate_step_workspace(int32_t rows, int32_t cols, size_t* bytes);
bmoe_status bmoe_substrate_step(int32_t rows, int32_t cols, const float* w, const void* o, double step, double decay,
                                float* w_out, uint32_t* packed, float* scale, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BMOE_UPDATE_H */
