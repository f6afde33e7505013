// What the linear layer's gradient needs of the multiply: two independent products in
// one launch, and the arrival counters that products use (defined in
// fp8_scaled_mm.hip; host code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8mm {

// out = bf16(scale_a[m] scale_b[n] sum_k A[m][k] B[n][k]), A in e5m2, B in e4m3fn.
struct Product {
    const void* A;
    const void* B;
    const float* scale_a;
    const float* scale_b;
    void* out;
    int64_t M, N, K;
};

struct PairPlan {
    int cfg;         // tile configuration of both, -1: two launches are the better plan
    int splits[2];
};

// Needs the sizes only.
PairPlan plan_pair(const Product (&p)[2]);

// Bytes of workspace of a plan with cfg >= 0.
int64_t pair_workspace(const Product (&p)[2], const PairPlan& plan);

// Arrival counters (32 bits each, from the workspace's start on) that have to be
// zero before a product of its own under the automatic plan, or before a pair.
int product_counters(const Product& p);
int pair_counters(const Product (&p)[2], const PairPlan& plan);

// An FP8MM_* status.  The pointers have been checked; `workspace` is as for
// fp8_scaled_mm_typed.
int run_pair(const Product (&p)[2], const PairPlan& plan, hipStream_t stream, void* workspace);

}  // namespace fp8mm
