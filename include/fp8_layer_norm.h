/*
 * fp8_layer_norm.h -- C ABI of the MI355X (gfx950) layer norm and its
 * gradient, with the float8 quantisation of the normalised rows.
 *
 * Forward, for each row of n = cols elements:
 *
 *     mean = sum(x) / n
 *     rstd = 1 / sqrt( sum((x - mean)^2) / n + eps )
 *     y    = (x - mean) * rstd * w + b
 *     scale = max|y| / qmax,  q = RNE( y / scale )      (row-wise, as fp8_quantize.h)
 *
 * Backward, with xh = (x - mean) * rstd and g = dy * w:
 *
 *     dx = rstd * ( g - sum(g) / n - xh * sum(g * xh) / n )  (+ residual_grad)
 *     dw = sum over rows of dy * xh,   db = sum over rows of dy
 *
 *   x, dy, y, residual_grad, dx   rows x cols, row-major (row stride cols), all
 *          of one type: bf16 or fp32.
 *   w, b   cols values, both fp32 or both bf16.  w NULL stands for ones, b
 *          NULL for zeros.
 *   mean, rstd   rows fp32 values.
 *   q      rows x cols float8 codes, scale rows fp32 values: what fp8_scaled_mm
 *          takes as A and scale_a.  The codes are made from the fp32 y, before
 *          y is rounded to its own type.
 *   dw, db cols fp32 values.
 *
 * Everything between the loads and the final rounding of an output is fp32.
 * Two calls with the same inputs give the same bits (no atomics in any sum).
 *
 * Rows that hold a NaN or an infinity: every y of the row is NaN, and so are rstd
 * and its scale, and its codes are NaN codes, so that a product made from them
 * shows it.  The same holds for rows of finite values whose sum, or whose sum of
 * (x - mean)^2, leaves the fp32 range (|x - mean| of about 1.8e19 / sqrt(n)).
 * With eps == 0 a row without variance has an infinite rstd and is NaN likewise.
 *
 * Pointers are DEVICE pointers on the current HIP device; the caller owns them
 * and the library keeps none after the call.  No entry point allocates,
 * memsets or synchronises: each enqueues kernels on `stream` (a hipStream_t;
 * NULL = default), so a call can be captured into a HIP graph.
 *
 * Preconditions (checked on the host before anything is enqueued):
 *   0 <= rows <= 2^31 - 1, 1 <= cols <= 2^24; cols % 16 == 0 where codes are
 *   asked for (the product reads whole 16-byte chunks).  Pointers aligned to
 *   their element; q 16-byte aligned.  Outputs must not overlap inputs or each
 *   other.  rows == 0: the forward call writes nothing, the backward call
 *   writes dw = db = 0; pointers to tensors without elements may be NULL.
 * Errors: FP8LN_OK (0) or an FP8LN_ERR_* code; on a validation error nothing is
 * enqueued.
 */
#ifndef FP8_LAYER_NORM_H
#define FP8_LAYER_NORM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct ihipStream_t;

enum fp8ln_dtype { FP8LN_BF16 = 0, FP8LN_FP32 = 1 };

/* formats of q: those of enum fp8mm_format */
enum fp8ln_format { FP8LN_E4M3FN = 0, FP8LN_E5M2 = 1 };

enum fp8ln_status {
    FP8LN_OK = 0,
    FP8LN_ERR_NULL = 1,      /* a required pointer is NULL */
    FP8LN_ERR_SHAPE = 2,     /* rows or cols out of range */
    FP8LN_ERR_ALIGN = 3,     /* a pointer is not aligned as required */
    FP8LN_ERR_DTYPE = 4,     /* unknown element type or code format */
    FP8LN_ERR_DEVICE = 5,    /* no usable HIP device */
    FP8LN_ERR_LAUNCH = 6,    /* the kernel launch failed */
    FP8LN_ERR_WORKSPACE = 7, /* workspace missing or too small */
    FP8LN_ERR_VALUE = 8      /* eps is negative or not finite */
};

/* Any of y, q (with scale) and the pair mean, rstd may be NULL: it is then not
 * written.  At least one of y and q is needed; q and scale come together, and
 * so do mean and rstd. */
int fp8_layer_norm(const void* x, int dtype, const void* w, const void* b, int param_dtype,
                   float eps, void* y, void* q, int q_format, float* scale, float* mean,
                   float* rstd, int64_t rows, int64_t cols, struct ihipStream_t* stream);

/* mean and rstd are the forward call's.  residual_grad (may be NULL) is the
 * gradient that reaches x along the residual path; it is added in fp32 before
 * dx is rounded.  `workspace` holds the workgroups' partial column sums: at
 * least fp8_layer_norm_backward_workspace_size(rows, cols) bytes, 256-byte
 * aligned, with any contents; it must not be used by two calls that can run at
 * the same time.  Calls on one stream may share it, from any host threads (the
 * launches of a call are enqueued without another's between them). */
int fp8_layer_norm_backward(const void* dy, const void* x, int dtype, const float* mean,
                            const float* rstd, const void* w, int param_dtype,
                            const void* residual_grad, void* dx, float* dw, float* db,
                            int64_t rows, int64_t cols, void* workspace, int64_t workspace_bytes,
                            struct ihipStream_t* stream);

/* Bytes of workspace that fp8_layer_norm_backward needs (host logic only; 0 for
 * an invalid problem or rows == 0). */
int64_t fp8_layer_norm_backward_workspace_size(int64_t rows, int64_t cols);

/* Static, NUL-terminated text for a status code. */
const char* fp8_layer_norm_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FP8_LAYER_NORM_H */
