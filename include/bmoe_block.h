/*
 * bmoe_block.h - from one block of a model to the next: the norm behind a block, its
 * gate, the scaled residual and the norm in front of the next block in one pass, forward
 * and backward.  (bmoe_norm.h has the plain layer norm of a residual stream.)
 *
 * For every row, with b the block's output (a ButterflyMoE layer's y, bmoe.h) and r the
 * residual stream in front of it
 *     z = N1(b) gamma_post + beta_post     (z = b without the norm behind the block)
 *     s = alpha r + scale gate z           (s = scale gate z without a residual)
 *     y = N2(s) gamma + beta
 * where N1 and N2 are of one kind:
 *     BMOE_NORM_LAYER: N(a) = (a - mean(a)) / sqrt(var(a) + eps),
 *     BMOE_NORM_RMS:   N(a) = a / sqrt(mean(a^2) + eps)  (beta, beta_post NULL).
 * gate is 1, one fp32 factor for each channel, or one of the activation dtype for each
 * token and channel.  z is not rounded; s is rounded to the activation dtype first and
 * N2 is that of the rounded row, so the backward, which reads the stored s, sees the
 * forward's values.  Statistics are fp32 sums over a row held in registers, as in
 * bmoe_norm.h: rows far from 0 and finite rows of any size (entries up to 2^127) are
 * normed as well as others (1 / deviation is infinite for deviations below 2^-128).
 *
 * Widths 1 .. 16384, rows 0 .. 2^24; arrays are row-major and dense, aligned to their
 * element size (16-byte alignment and a width that is a multiple of 8 are fastest).
 * Memory rules as in bmoe.h: every pointer is caller-owned device memory, nothing is
 * allocated or synchronised, all work is enqueued on `stream`, results do not depend on
 * scheduling, and all errors but BMOE_ERR_HIP are found before anything is enqueued.
 */
#ifndef BMOE_BLOCK_H
#define BMOE_BLOCK_H

#include "bmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BMOE_NORM_LAYER = 0, BMOE_NORM_RMS = 1 } bmoe_norm_kind;
typedef enum { BMOE_GATE_NONE = 0, BMOE_GATE_CHANNEL = 1, BMOE_GATE_ROWS = 2 } bmoe_gate_kind;

/* What forward and backward of one place in a model have in common. */
typedef struct bmoe_block_norm {
  int32_t rows, width;
  int32_t dtype;            /* bmoe_dtype of b, r, s, y, a gate of rows and their gradients */
  int32_t kind;             /* bmoe_norm_kind */
  int32_t post;             /* 1: with the norm behind the block, 0: z = b */
  int32_t gate_kind;        /* bmoe_gate_kind */
  float alpha, scale;       /* finite */
  float eps;                /* finite, not negative */
  int32_t reserved;         /* 0 */
  const void* gate;         /* [width] fp32 (channel), [rows][width] of dtype (rows), NULL (none) */
  const float* gamma_post;  /* [width] or NULL (ones; NULL with post 0) */
  const float* beta_post;   /* [width] or NULL (zeros; NULL with post 0 and for RMS) */
  const float* gamma;       /* [width] or NULL (ones) */
  const float* beta;        /* [width] or NULL (zeros; NULL for RMS); unused in the backward */
} bmoe_block_norm;

/* Forward.
 *   b       [rows][width], read only.
 *   r       [rows][width] or NULL, read only.
 *   s       [rows][width], written; may be the same buffer as r, or as b where no
 *           backward follows.
 *   y       [rows][width], written; may be the same buffer as b or r where that one is not
 *           needed any more (not as s).
 *   stats   [rows][4] fp32 (16-byte aligned), written with mean and 1 / deviation of b
 *           (0, 0 with post 0; mean 0 for RMS), then those of s, for the backward; or NULL.
 * A row that holds a NaN or an infinity becomes NaN, other rows are not affected.
 * Errors: BMOE_ERR_NULL, BMOE_ERR_SHAPE, BMOE_ERR_DTYPE (dtype, kind, gate_kind),
 * BMOE_ERR_ALIGN, BMOE_ERR_ALIAS, BMOE_ERR_DEVICE, BMOE_ERR_HIP. */
bmoe_status bmoe_block_norm_forward(const bmoe_block_norm* n, const void* b, const void* r, void* s, void* y,
                                    float* stats, hipStream_t stream);

/* Gradients of a weight; each may be NULL (not wanted).  fp32 [width], sums over all
 * rows, zero for rows = 0; gate: fp32 [width] (channel) or [rows][width] of dtype (rows).
 * One that the forward has no use for (beta for RMS, post's without it, gate without one) is
 * NULL. */
typedef struct bmoe_block_norm_grads {
  float* gamma_post;
  float* beta_post;
  void* gate;
  float* gamma;
  float* beta;
} bmoe_block_norm_grads;

/* Device workspace bytes of bmoe_block_norm_backward (partial sums of the weights'
 * gradients; the same for every set of gradients wanted). */
bmoe_status bmoe_block_norm_backward_workspace(const bmoe_block_norm* n, size_t* bytes);

/* Backward at the forward's s and stats.
 *   dy        [rows][width] of dy_dtype: fp32 (the input gradient of bmoe_layer_backward)
 *             or dtype, read only.
 *   b, s, stats   of the forward, read only.
 *   d_sum     [rows][width] of dtype or NULL: gradient that reaches s past N2 (the
 *             residual stream's own), read only.
 *   db        [rows][width] of dtype, written; may be the same buffer as b, s or d_sum, or
 *             as dy when dy_dtype is dtype.
 *   dr        [rows][width] of dtype, written, or NULL (no residual); may be the same
 *             buffer as any of those that db may be, but not as db.
 *   grads     what is wanted of the weights' gradients, or NULL.
 *   workspace at least bmoe_block_norm_backward_workspace bytes, 16-byte aligned,
 *             contents undefined after; may be NULL when no [width] gradient is wanted.
 * With ds the gradient of s: dr = alpha ds, gate: scale z ds, db: N1's backward of scale
 * gate ds.  Column sums are fp32, added in an order that the sizes alone decide.  Errors
 * as above, and BMOE_ERR_WORKSPACE. */
bmoe_status bmoe_block_norm_backward(const bmoe_block_norm* n, int32_t dy_dtype, const void* dy, const void* b,
                                     const void* s, const float* stats, const void* d_sum, void* db, void* dr,
                                     const bmoe_block_norm_grads* grads, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BMOE_BLOCK_H */
