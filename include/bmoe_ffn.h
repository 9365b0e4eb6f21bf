/*
 * bmoe_ffn.h - the dense gated feed-forward block, forward and backward: what a model
 * has in its layers without experts, and beside a ButterflyMoE layer (bmoe.h) where some
 * of the work is every token's (a shared expert, added to what the routed ones give).
 *
 *     g = x Wg^T,  u = x Wu^T,  h = act(g) u,  y = h Wd^T (+ add)
 * with act(g) = g / (1 + exp(-g)) (BMOE_GATED_SILU) or g Phi(g) (BMOE_GATED_GELU, the exact
 * GELU), Wg and Wu [ff][d], Wd [d][ff].  Both projections, the activation and the product
 * are one kernel.  All matrices are bf16 and row-major; products run on the matrix cores
 * with fp32 sums, g and u stay fp32 up to h, which is rounded to bf16 (with up to 4 tokens,
 * which do without matrix cores, only for the state: the same token's y differs in its last
 * bits between a batch of 4 and one of 5), as are the backward's dg and du; their factors
 * u act'(g) and act(g) are kept to 12 significant bits.  Sums' orders, and with them last
 * bits, go by the sizes of a call.
 *
 * tokens 0 .. 2^24; d and ff positive multiples of 8, d <= 16384, ff <= 65536, d ff <= 2^29,
 * tokens * max(d, ff) <= 2^36.  Memory rules as in bmoe.h: every pointer is caller-owned
 * device memory, 16-byte aligned, nothing is allocated or synchronised, all work is
 * enqueued on `stream`, results do not depend on scheduling, and all errors but
 * BMOE_ERR_HIP are found before anything is enqueued.  Calls that may overlap in time
 * need workspaces and outputs of their own.
 */
#ifndef BMOE_FFN_H
#define BMOE_FFN_H

#include "bmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BMOE_GATED_SILU = 0, BMOE_GATED_GELU = 1 } bmoe_gated_act;

/* What a backward reads of the forward, 7 bytes for each token and hidden unit: h and the two
 * factors. */
bmoe_status bmoe_gated_ffn_state_size(int32_t tokens, int32_t ff, size_t* bytes);

/* Forward.
 *   x        [tokens][d], read only.
 *   w_in     [2 ff][d], Wg above Wu, read only.
 *   w_down   [d][ff], read only.
 *   add      [tokens][d] or NULL, read only.
 *   y        [tokens][d], written; may be the same buffer as add.
 *   state    bmoe_gated_ffn_state_size bytes, written, for the backward; or NULL.
 *   workspace at least bmoe_gated_ffn_forward_workspace bytes, contents undefined after;
 *            may be NULL when that is 0.  with_state: whether state is given.
 * Errors: BMOE_ERR_SHAPE, BMOE_ERR_DTYPE (act), BMOE_ERR_NULL, BMOE_ERR_ALIGN,
 * BMOE_ERR_ALIAS, BMOE_ERR_WORKSPACE (also a state of fewer bytes), BMOE_ERR_DEVICE,
 * BMOE_ERR_HIP. */
bmoe_status bmoe_gated_ffn_forward_workspace(int32_t tokens, int32_t d, int32_t ff, int32_t with_state, size_t* bytes);
bmoe_status bmoe_gated_ffn_forward(int32_t tokens, int32_t d, int32_t ff, int32_t act, const void* x, const void* w_in,
                                   const void* w_down, const void* add, void* y, void* state, size_t state_bytes,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Backward of sum(dy y), at the forward's state, which is read only.
 *   act      one of the activations; the gradients are those of the state's own, whose
 *            slopes it holds, whichever is given here.
 *   dy       [tokens][d], read only.
 *   dx_add   [tokens][d] fp32 or NULL, read only: added into dx before it is rounded (the
 *            input gradient of bmoe_layer_backward for the same x).
 *   dx       [tokens][d] bf16, written, or NULL (not wanted).
 *   dw_in    [2 ff][d] bf16, written, or NULL; dw_down [d][ff] bf16, written, or NULL: sums
 *            over all tokens, zero for tokens = 0.
 *   workspace at least bmoe_gated_ffn_backward_workspace bytes, contents undefined after.
 * (The gradient of add is dy.)  Errors as above. */
bmoe_status bmoe_gated_ffn_backward_workspace(int32_t tokens, int32_t d, int32_t ff, size_t* bytes);
bmoe_status bmoe_gated_ffn_backward(int32_t tokens, int32_t d, int32_t ff, int32_t act, const void* x, const void* w_in,
                                    const void* w_down, const void* dy, const void* state, size_t state_bytes,
                                    const float* dx_add, void* dx, void* dw_in, void* dw_down, void* workspace,
                                    size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BMOE_FFN_H */
