/*
 * bmoe_adamw.h - one AdamW step over many tensors: the rotation angles, the gate
 * matrix and the norm weights of ButterflyMoE layers (bmoe_layer_backward of
 * bmoe_train.h leaves their gradients; the latent substrates have their own step in
 * bmoe_update.h), or any other tensors.
 *
 * For every value, with the gradient g times *grad_scale where that is given, and t
 * the number of this step (1, 2, ..)
 *     m' = beta1 m + (1 - beta1) g,   v' = beta2 v + (1 - beta2) g^2
 *     p' = (1 - lr_t decay) p - lr_t (m' / (1 - beta1^t)) / (sqrt(v' / (1 - beta2^t)) + eps)
 * where lr_t = lr lr_scale.  All in fp32; p, m, v are updated in place and `copy`,
 * where given, gets p' rounded to bf16.  Infinities and NaNs go through these
 * formulas as they are and stay in their value.  With an eps of 0, a v' of 0 (g^2 below
 * fp32's smallest number) makes p' infinite, or NaN where m' is 0 too.
 *
 * Moments in 8 bits.  Blocks of 256 consecutive values share a power of two for m and
 * one for v, and each value has a code of 8 steps to a factor of two:
 *     m: sign bit, then code c of |m|, v: code c of v, and with k = max(c / 8 - 1, 0)
 *     the value (c - 8 k) 2^(k + e - top - 3),   top = 13 for m, 29 for v,
 * e the exponent of the block's largest finite value (2^e <= it < 2^(e + 1), e in
 * [-126, 127]), stored as the byte e + 127.  So m reaches 2^-17 of its block's largest
 * value and v 2^-33.  Codes 127 of m and 255 of v are NaN (and stand for
 * infinities), and no finite value takes the code of 2^128.  A v that is not 0 never gets
 * code 0: its value stays the divisor.
 * p' is that of m' and v' before they become codes.  A value between two codes takes the
 * upper one with a probability that makes the expected value right (v changes by
 * 1 - beta2 of itself a step, a hundredth of the codes' distance: rounded to the
 * nearest it would stay where it is), by 16 bits each of
 *     mix(i 0x9E3779B1 + (i >> 32) 0xBB67AE85 + key),   the lower ones for m,
 *     key = mix(t 0x9E3779B1 + mix(index 0xBB67AE85 + seed)),
 *     mix(h): h = (h ^ h >> 15) 0x6A09E667, h = (h ^ h >> 13) 0x3C6EF373, h ^ h >> 16,
 * all modulo 2^32, i the value's place in its tensor and index the tensor's in the
 * call: the same inputs give the same codes.
 *
 * Memory rules as in bmoe.h: every pointer in the tensors is caller-owned device
 * memory, nothing is allocated or synchronised, all work is enqueued on `stream`,
 * results do not depend on scheduling, and all errors but BMOE_ERR_HIP are found
 * before anything is enqueued.  The arrays `tensors` and `args` are host memory, read
 * before the call returns.
 */
#ifndef BMOE_ADAMW_H
#define BMOE_ADAMW_H

#include "bmoe.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BMOE_ADAMW_BLOCK 256

typedef struct bmoe_adamw_tensor {
  float* param;          /* [n], updated */
  const void* grad;      /* [n] of grad_dtype, read; NULL: the tensor is left as it is */
  void* m;               /* [n] fp32, or codes (one byte each), updated */
  void* v;               /* the same */
  uint8_t* m_exp;        /* [ceil(n / 256)], updated, with 8 bits; else NULL */
  uint8_t* v_exp;        /* the same */
  void* copy;            /* [n] bf16, written, or NULL */
  int64_t n;             /* 0 .. 2^33 */
  float lr_scale;        /* finite */
  float weight_decay;    /* finite */
  int32_t grad_dtype;    /* bmoe_dtype */
  int32_t bits;          /* of the moments: 32 or 8 */
} bmoe_adamw_tensor;

typedef struct bmoe_adamw_args {
  double lr;                  /* finite; unused with lr_device */
  double beta1, beta2;        /* in [0, 1) */
  double eps;                 /* 0 or in [2^-126, 2^126] */
  int64_t step;               /* t, at least 1; unused with step_device */
  int64_t* step_device;       /* 1 value on the device or NULL: the steps taken before,
                                 raised by 1 first; a captured call counts on in every replay */
  const float* lr_device;     /* 1 value on the device or NULL */
  const float* grad_scale;    /* 1 value on the device or NULL */
  uint32_t seed;
  uint32_t reserved;          /* 0 */
} bmoe_adamw_args;

/* One step.  Arrays of fp32 are 4-byte aligned, bf16 ones 2-byte, step_device 8-byte
 * (16-byte alignment of all of a tensor's arrays, 8 of bf16 ones and 4 of codes, is
 * fastest).  Nothing that is written may overlap anything else, in one tensor or in
 * two.  Errors: BMOE_ERR_NULL, BMOE_ERR_SHAPE, BMOE_ERR_DTYPE (grad_dtype, bits),
 * BMOE_ERR_ALIGN, BMOE_ERR_ALIAS, BMOE_ERR_DEVICE, BMOE_ERR_HIP. */
bmoe_status bmoe_adamw_step(const bmoe_adamw_tensor* tensors, int32_t count, const bmoe_adamw_args* args,
                            hipStream_t stream);

/* The values of 8-bit moments: m_out[i] and v_out[i] [n] of out_dtype (bmoe_dtype; a step's
 * codes are exact in either, in bf16 from 2^-130 on, below which its numbers are 2^-133
 * apart and take the nearest) for tensor i, either of them NULL if not wanted
 * (param, grad and copy are not used).  m_out and v_out are host arrays of `count`
 * device pointers.  Errors as above; BMOE_ERR_DTYPE for bits other than 8. */
bmoe_status bmoe_adamw_moments(const bmoe_adamw_tensor* tensors, int32_t count, int32_t out_dtype, void* const* m_out,
                               void* const* v_out, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* BMOE_ADAMW_H */
