// A weight's codes in both layouts for gfx950 (MI355X) (formulas and contract:
// include/fp8_quantize_weight.h; kernels: column_codes.h).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8_quantize_weight.h"
#include "column_codes.h"
#include "enqueue_lock.h"

namespace {

bool at(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int64_t kMaxRows = int64_t(1) << 27, kMaxCols = int64_t(1) << 23;

int weight_shape(int64_t N, int64_t K) {
    if (N < 0 || N > kMaxRows || K < 16 || K > kMaxCols || K % 16 != 0 || !code_grid_ok(N, K))
        return FP8MM_ERR_SHAPE;
    return FP8MM_OK;
}

CodeJob weight_job(int64_t N, int64_t K) {
    CodeJob p{};
    p.M = N;
    p.K = K;
    p.Mp = code_up(N, 16) * 16;
    p.col_unit = 1.f;
    plan_codes(p);
    return p;
}

__global__ void __launch_bounds__(256) zero_floats_kernel(float* p, int64_t n) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = 0.f;
}

template <class T, int FMT>
void launch_weight(const CodeJob& p, hipStream_t hs) {
    if (p.M * p.K * (int64_t)sizeof(T) > kCachedBytes && sizeof(T) == 2) launch_codes<T, FMT, true, sizeof(T) == 2>(p, NoFactor(), hs);
    else launch_codes<T, FMT, true, false>(p, NoFactor(), hs);
}

}  // namespace

extern "C" {

int64_t fp8_quantize_weight_workspace_size(int64_t N, int64_t K) {
    return weight_shape(N, K) != FP8MM_OK ? -1 : code_partials(weight_job(N, K), true);
}

int fp8_quantize_weight(const void* w, int dtype, int format, void* q, float* scale, void* qt, float* scale_t,
                        int64_t N, int64_t K, struct ihipStream_t* stream, void* workspace,
                        int64_t workspace_bytes) {
    if ((dtype != FP8W_BF16 && dtype != FP8W_FP32) || (format != FP8MM_E4M3FN && format != FP8MM_E5M2))
        return FP8MM_ERR_FORMAT;
    int st = weight_shape(N, K);
    if (st != FP8MM_OK) return st;
    if (!scale_t || (N > 0 && (!w || !q || !scale || !qt))) return FP8MM_ERR_NULL;
    if (!at(w, dtype == FP8W_BF16 ? 2 : 4) || !at(q, 16) || !at(qt, 16) || !at(scale, 4) || !at(scale_t, 4) ||
        !at(workspace, 256))
        return FP8MM_ERR_ALIGN;
    CodeJob p = weight_job(N, K);
    if (N > 0 && (!workspace || workspace_bytes < code_partials(p, true))) return FP8MM_ERR_WORKSPACE;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return FP8MM_ERR_DEVICE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (N == 0) {
        hipLaunchKernelGGL(zero_floats_kernel, dim3(64), dim3(256), 0, hs, scale_t, K);
        return hipGetLastError() == hipSuccess ? FP8MM_OK : FP8MM_ERR_LAUNCH;
    }
    std::lock_guard<std::mutex> together(fp8mm::enqueue_lock(workspace));
    p.x = w;
    p.col_max = static_cast<float*>(workspace);
    p.row_max = p.col_max + (int64_t)p.parts * K;
    p.col_scale = scale_t;
    p.row_scale = scale;
    p.q_rows = static_cast<uint8_t*>(q);
    p.q_cols = static_cast<uint8_t*>(qt);
    if (dtype == FP8W_BF16) {
        if (format == FP8MM_E4M3FN) launch_weight<bf16_t, 0>(p, hs);
        else launch_weight<bf16_t, 1>(p, hs);
    } else {
        if (format == FP8MM_E4M3FN) launch_weight<float, 0>(p, hs);
        else launch_weight<float, 1>(p, hs);
    }
    return hipGetLastError() == hipSuccess ? FP8MM_OK : FP8MM_ERR_LAUNCH;
}

}  // extern "C"
