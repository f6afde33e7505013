/*
 * adamw.h -- C ABI of the MI355X (gfx950) AdamW step over many tensors at once, with
 * moments of 32 or 8 bits.
 *
 * For each element (decay apart from the gradient; Loshchilov and Hutter, "Decoupled
 * weight decay regularization"), with g the gradient times *grad_scale:
 *
 *     m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *     p = p (1 - lr weight_decay)
 *           - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 *
 *   in fp32 (1 - beta and 1 - beta^step in fp64, then rounded); in m, v and sqrt(v) every
 *   product, sum and root is rounded as it is written.  The step's quotient is fp32's with
 *   moments of 32 bits, with 8 a product by the hardware's reciprocal (off by 2^-22 of
 *   itself at most); an eps above 0 counts as 2^-149 at least, as 2^-126 with 8 bits.  p
 *   is the master weight where there is one; the parameter is then p rounded to bf16.  A bf16
 *   parameter without a master is rounded to nearest, so steps below half its last bit
 *   leave it as it is.
 *
 * Moments of 8 bits.  A tensor is cut into blocks of 256 elements, the last one
 * shorter.  exp_avg holds e4m3fn codes of m over the block's scale, max |m| / 448;
 * exp_avg_sq those of sqrt(v) (half the exponents that v would need) over its own.
 * A scale below 2^-100 is 0, with codes 0.  The step computes with the stored values,
 * updates p with the new ones in fp32 and rounds those at random to one of the two
 * neighbouring codes, up with the probability of the part of the step that is left
 * (rounded to nearest, a moment that moves by a thousandth of itself would never move
 * in 3 bits): up where r / 2^16 and that part make a whole one, r the low 16 bits (m) or the
 * high ones (sqrt(v)) of h for the element's position.  sqrt(v) > 0 is never rounded to 0, which
 * would leave eps alone under m.  With all arithmetic modulo 2^32, and n the element's
 * place in its tensor plus 256 times the blocks of the tensors before it in the call,
 *
 *     h0 = n 0x6A09E667 + seed 0xBB67AE85,       h1 = (h0 ^ h0 >> 15) 0x3C6EF373,
 *     h2 = (h1 ^ h1 >> 13) 0xA54FF53B,           h  = h2 ^ h2 >> 16
 *
 *   so calls of equal arguments give equal bits; the seed should differ from step to
 *   step.
 *
 * A NaN or an infinity of the gradient shows in its element's outputs; in 8 bits an
 * infinity also takes its block's other moments (their scale is infinite).
 */
#ifndef ADAMW_H
#define ADAMW_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t; /* hipStream_t is `struct ihipStream_t*` */

enum adamw_dtype { ADAMW_BF16 = 0, ADAMW_FP32 = 1 };

enum adamw_status {
    ADAMW_OK = 0,
    ADAMW_ERR_NULL = 1,   /* a required pointer is NULL, or one that has to be is not */
    ADAMW_ERR_SHAPE = 2,  /* a negative size, or too many elements */
    ADAMW_ERR_ALIGN = 3,  /* a pointer is not aligned to its element */
    ADAMW_ERR_DTYPE = 4,  /* unknown type, or a master of fp32 parameters */
    ADAMW_ERR_VALUE = 5,  /* lr, betas, eps, weight_decay or step out of range */
    ADAMW_ERR_DEVICE = 6, /* no usable HIP device */
    ADAMW_ERR_LAUNCH = 7, /* a kernel launch failed */
    ADAMW_ERR_ALIAS = 8   /* parameters or their states overlap */
};

/* One tensor: device pointers.  exp_avg and exp_avg_sq are fp32, or codes; the scales
 * (one for each block) belong to 8 bits, master may be NULL. */
struct adamw_tensor {
    void* param;
    const void* grad;
    void* exp_avg;
    void* exp_avg_sq;
    float* master;
    float* exp_avg_scale;
    float* exp_avg_sq_scale;
    int64_t numel;
};

/* Numbers of the step.  Each pointer (device, one element) takes the place of the
 * value beside it where it is not NULL: for a captured step, whose values change from
 * replay to replay.  lr and weight_decay are at least 0, betas in [0, 1), eps at least
 * 0, all finite; step counts from 1. */
struct adamw_numbers {
    double lr, beta1, beta2, eps, weight_decay;
    int64_t step;
    uint32_t seed;
    const float* lr_ptr;
    const float* step_ptr;
    const int64_t* seed_ptr;
    const float* grad_scale_ptr;   /* NULL: 1 */
};

/* One step over `count` tensors, `tensors` being a host array that the call has read
 * when it returns.  All parameters have one type, all gradients one, all states
 * state_bits (8 or 32); either every tensor has a master or none has.  Parameters,
 * masters, moments and scales are written in place, of any sizes (0 included) and
 * alignment above their element's; two of them must not overlap (ADAMW_ERR_ALIAS), nor one a gradient
 * (which is not checked; one gradient may be several tensors').
 * Asynchronous on `stream`, one launch for each 48 tensors; nothing is allocated, so it
 * may be captured.  On an error nothing is enqueued (ADAMW_ERR_LAUNCH aside). */
int adamw_step(const struct adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype,
               int state_bits, const struct adamw_numbers* numbers, struct ihipStream_t* stream);

/* Static, NUL-terminated text for a status code. */
const char* adamw_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* ADAMW_H */
