// What the cross entropy needs of the multiply: products whose epilogue makes
// softmax statistics or the codes of the logits' gradient, and a product whose K
// range comes in pieces (defined in fp8_scaled_mm.hip; host code).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_pair.h"

namespace fp8mm {

// z[m][j] = s sum_k A[m][k] B[j][k], as in fp8_scaled_mm_typed.
struct Logits {
    const void* A;
    int a_format;
    const void* B;
    int b_format;
    const float* scale_a;
    const float* scale_b;
    int64_t M, V, K;
    int mode;
};

struct LossPlan {
    int cfg, splits;
};

// Needs the sizes only.
LossPlan loss_plan(int64_t M, int64_t V, int64_t K);
// Whether the plan's work units can be counted in an int.
bool loss_plan_fits(int64_t M, int64_t V, const LossPlan& plan);
// Column blocks that a row's statistics come in.
int64_t loss_blocks(int64_t V, const LossPlan& plan);
// Rows that the plan's tiles cover, M or more.
int64_t loss_rows(int64_t M, const LossPlan& plan);
// Bytes of workspace (arrival counters first), and how many counters of 32 bits
// have to be zero before the launch.
int64_t loss_workspace(int64_t M, int64_t V, const LossPlan& plan);
int loss_counters(int64_t M, int64_t V, const LossPlan& plan);

// Where the ping-pong kernel takes a product of `fixed` rows (or columns) by `n`
// columns (or rows) over k bytes, and the last of its rounds over the CUs would leave
// most of them idle: how many of the n belong in a launch of whole rounds, the others
// in one of their own (smaller tiles).  Else n.
int64_t whole_rounds(int64_t fixed, int64_t n, int64_t k);
// Work units of a tile, for run_sum, of a product over a long k (0: the automatic plan
// of fp8_scaled_mm_typed is as good).
int long_sum_splits(int64_t M, int64_t N, int64_t k);
int ping_pong_config();

// Each enqueues one launch and returns an FP8MM_* status; the pointers have been
// checked.
int run_stats(const Logits& z, const LossPlan& plan, const int64_t* target, float2* part, int64_t col0,
              hipStream_t stream, void* workspace);
int run_codes(const Logits& z, const LossPlan& plan, const float2* rows, uint8_t* q, int64_t ldq, uint8_t* qt,
              int64_t ldqt, int64_t col0, hipStream_t stream, void* workspace);

// The product under its automatic plan, its output kept out of the caches from 128 MB on
// (which hold what the caller's next launches read).
int run_streamed(const Product& p, hipStream_t stream, void* workspace, int64_t workspace_bytes);

// One piece of out = bf16(scale_a[m] scale_b[n] sum_k A[m][k] B[n][k]): K of it in
// this call, A in e5m2 with rows K apart, rows of B ldb apart.  With splits > 1 there is
// one piece only, whose tiles take that many work units each, joined by a second launch.
struct SumPiece {
    const void* A;
    const void* B;
    int b_format;
    const float* scale_a;
    const float* scale_b;
    void* out;
    int64_t M, N, K, ldb;
    bool first, last;
    int splits;
};
int64_t sum_workspace(int64_t M, int64_t N, int splits);
int run_sum(const SumPiece& p, hipStream_t stream, void* sums);

}  // namespace fp8mm
