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

#ifdef __cplusplus
}
#endif

#endif /* FP8_LINEAR_H */
