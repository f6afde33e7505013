/*
 * fp8_linear.h -- C ABI of the MI355X (gfx950) FP8 linear layer: the scaled
 * multiply with bias, activation and residual in its epilogue, and its
 * gradient.
 *
 * Forward (s, A, B, bias and the operand formats as in fp8_scaled_mm.h):
 *
 *     z[m][n]      = s[m][n] * sum_{k<K} A[m][k] * B[n][k]  (+ bias[n])
 *     out[m][n]    = bf16_rne( act(z[m][n])  (+ residual[m][n]) )
 *     preact[m][n] = bf16_rne( z[m][n] )                      (optional)
 *
 *   act  FP8MM_ACT_NONE z, _RELU max(z, 0), _GELU z Phi(z) (Phi the normal
 *        distribution function), _GELU_TANH z sigmoid(2 u) with
 *        u = sqrt(2/pi) (z + 0.044715 z^3), _SILU z sigmoid(z).
 *   z, act(z) and the residual's addition are fp32; each output is rounded
 *   once.  preact is what the gradient takes.
 */
#ifndef FP8_LINEAR_H
#define FP8_LINEAR_H

#include <stdint.h>

#include "fp8_scaled_mm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum fp8mm_activation {
    FP8MM_ACT_NONE = 0,
    FP8MM_ACT_RELU = 1,
    FP8MM_ACT_GELU = 2,
    FP8MM_ACT_GELU_TANH = 3,
    FP8MM_ACT_SILU = 4
};

/* fp8_scaled_mm_typed with the epilogue above: the same operands, plans
 * (config_id, splits), workspace (fp8_scaled_mm_workspace_size), execution,
 * preconditions and status codes.  residual and preact are M x N bf16,
 * row-major, 2-byte aligned, and may be NULL; `out` may be the residual's own
 * memory, and must not overlap anything else.  FP8MM_ERR_ACTIVATION for an
 * unknown activation, FP8MM_ERR_CONFIG for a stream-K plan where any of
 * activation, residual and preact is asked for. */
int fp8_linear(const void* A, int a_format, const void* B, int b_format, const float* scale_a,
               const float* scale_b, const void* bias_or_null, const void* residual_or_null,
               int activation, void* preact_or_null, void* out, int64_t M, int64_t N, int64_t K,
               int scaling_mode, struct ihipStream_t* stream, int config_id, int splits,
               void* workspace, int64_t workspace_bytes);

/* The gradient of out = act(x W^T + bias) with float8 operands.  For dy, the
 * gradient of act(z), and z = preact of the forward call:
 *
 *     dz    = dy * act'(z)                           (fp32)
 *     dbias = sum over rows of dz                    (fp32)
 *     dx    = bf16_rne( dz W ):    dz as e5m2 with one scale for each row
 *     dw    = bf16_rne( dz^T x ):  dz as e5m2 with one scale for each column,
 *                                  x as e4m3fn with one scale for each column
 *
 *   Scales are max / qmax (57344, 448) and codes RNE(value / scale), as in
 *   fp8_quantize.h: for dz of none and relu and for x (values of few bits, whose
 *   quotients meet ties) with the correctly rounded quotient, for the other
 *   activations with the product by 1 / scale.  A row or column whose scale
 *   would be below 2^-126 has scale 0 and codes 0.
 *
 *   dy, z  M x N bf16;  x  M x K bf16 (row-major).  z may be NULL for
 *          FP8MM_ACT_NONE.  (dy also is the residual's gradient.)
 *   wt     W transposed: K x N float8 codes of wt_format, row-major, with
 *          wt_scale[k] for row k, laid out once for each update of the weights.
 *   dx     M x K bf16, dw  N x K bf16, dbias  N fp32.  Each may be NULL: what
 *          only it needs is then not computed (x, and wt with its scales, may
 *          then be NULL too).  At least one of them is needed.
 *
 * A NaN in dz or x comes out in the outputs that it reaches, and so does an
 * infinity (as a NaN).
 * Preconditions: 0 <= M <= 2^31 - 1, 16 <= N, K <= 2^23, both multiples of 16;
 * with dw also M <= 2^23.  wt 16-byte aligned, bf16 tensors 2-byte, fp32 ones
 * 4-byte aligned.  Outputs must not overlap inputs or each other.  With M == 0, dw and dbias are zeros.
 * `workspace` is 256-byte aligned, of any contents, and at least
 * fp8_linear_backward_workspace_size() bytes (the first 256 KiB of it are arrival
 * counters, which the call clears).  It may serve calls of any shape, one at a
 * time: those of one stream, from any host threads (the launches of a call are
 * enqueued without another's between them).  Execution and status codes are those of
 * fp8_scaled_mm.h; equal calls give equal bits (what else a call asks for may
 * change the plan, and with it the order of an output's fp32 sums). */
int fp8_linear_backward(const void* dy, const void* x_or_null, const void* wt_or_null,
                        int wt_format, const float* wt_scale_or_null, const void* z_or_null,
                        int activation, void* dx_or_null, void* dw_or_null, float* dbias_or_null,
                        int64_t M, int64_t N, int64_t K, struct ihipStream_t* stream,
                        void* workspace, int64_t workspace_bytes);

/* Bytes of workspace for the outputs asked for (host logic only; -1 for an
 * invalid problem). */
int64_t fp8_linear_backward_workspace_size(int64_t M, int64_t N, int64_t K, int want_dx,
                                           int want_dw);

#ifdef __cplusplus
}
#endif

#endif /* FP8_LINEAR_H */
