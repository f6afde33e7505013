/*
 * fp8_quantize_weight.h -- C ABI of the MI355X (gfx950) quantisation of a weight into
 * the two layouts that products take it in: N x K with one scale for each row (the
 * forward product's B) and, transposed, K x Np with one scale for each column of w
 * (the gradient's wt, fp8_linear.h and fp8_cross_entropy.h).
 *
 *     scale[n]   = max_k |w[n][k]| / qmax,   q[n][k]  = RNE(clamp(w[n][k] / scale[n]))
 *     scale_t[k] = max_n |w[n][k]| / qmax,   qt[k][n] = RNE(clamp(w[n][k] / scale_t[k]))
 *
 *   qmax is 448 (FP8MM_E4M3FN) or 57344 (FP8MM_E5M2).  Scales are fp32, quotients the
 *   correctly rounded fp32 ones, as in fp8_quantize.h: of a bf16 w, both outputs have
 *   the bits that fp8_quantize_* gives of w and of its transpose.  A row or column of
 *   zeros has scale 0 and codes 0; a NaN is skipped by the maxima and comes out as a
 *   NaN code; with an infinity the scale is infinite, its code a NaN and the others 0.
 *
 *   w        N x K, row-major, bf16 or fp32.
 *   q, qt    N x K and K x Np codes, row-major; Np = N rounded up to 16, codes 0 past N.
 *   scale    N fp32,  scale_t  K fp32.
 *
 * All pointers are device pointers of the current device; the library keeps none.
 * Execution is asynchronous on `stream`, nothing is allocated, and every call may be
 * captured.  Preconditions (checked before anything is enqueued): 0 <= N <= 2^27,
 * 16 <= K <= 2^23, K % 16 == 0, at most 2^24 - 1 tiles of 128 x 128; w aligned to its
 * element, q and qt to 16 bytes, scales to 4; outputs overlap nothing.  With N == 0
 * only scale_t (zeros) is written.  `workspace` is 256-byte aligned, of any contents,
 * and at least fp8_quantize_weight_workspace_size() bytes; it may serve calls of any
 * shape, one at a time (those of one stream, from any host threads).
 * Returns FP8MM_OK or an FP8MM_ERR_* of fp8_scaled_mm.h (FP8MM_ERR_FORMAT also for an
 * unknown dtype).
 */
#ifndef FP8_QUANTIZE_WEIGHT_H
#define FP8_QUANTIZE_WEIGHT_H

#include <stdint.h>

#include "fp8_scaled_mm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum fp8_weight_dtype { FP8W_BF16 = 0, FP8W_FP32 = 1 };

int fp8_quantize_weight(const void* w, int dtype, int format, void* q, float* scale, void* qt, float* scale_t,
                        int64_t N, int64_t K, struct ihipStream_t* stream, void* workspace,
                        int64_t workspace_bytes);

/* Bytes of workspace (host logic only; -1 for an invalid problem). */
int64_t fp8_quantize_weight_workspace_size(int64_t N, int64_t K);

#ifdef __cplusplus
}
#endif

#endif /* FP8_QUANTIZE_WEIGHT_H */
