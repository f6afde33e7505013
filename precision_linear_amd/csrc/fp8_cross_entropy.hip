// The softmax cross entropy of an FP8 linear layer and its gradient for gfx950
// (MI355X) (formulas: include/fp8_cross_entropy.h).
//
// Forward: the multiply's kernels with an epilogue that reduces each tile's logits
// to the largest and the sum of exponentials of each row (by tiles, in the ping-pong
// kernel by the 64 columns of a wave), the target's left out; loss_kernel joins them
// with the target's logit, which it makes itself in fp32: the matrix instruction keeps a product
// to 2^-13 of its largest, which averages out among the others.  The loss is log(1 +
// sum of the others over the target's), so that a row that is sure of its target keeps
// what little is left.  The product bounds it: 8 bytes leave the multiply for 64 logits.
//
// Gradient: the logits once more, with an epilogue that turns them into e5m2 codes
// of dz, written by rows (for dx) and by columns (for dw), then the two products.
// The row's scale is known beforehand (the target's element is a row's largest), and
// the row's factor r = dloss h goes to the other operand of dw, so one set of codes
// serves both products.  The vocabulary comes in pieces of 256 entries or
// more that keep the codes in kCodeBytes of workspace (up to 2^20 rows; beyond, 256 entries take 512
// bytes a row, 4 GiB at 2^23); dx's fp32 sums stay in 256 x 256 tiles of the accumulators' own
// layout from piece to piece (1 KiB for each row and 256 columns begun).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/fp8_cross_entropy.h"
#include "activation.h"
#include "column_codes.h"
#include "enqueue_lock.h"
#include "fp8_loss.h"
#include "fp8_pair.h"

namespace {

constexpr int kLossThreads = 1024;
constexpr float kE5m2Max = 57344.f, kLog2E5m2Max = 15.807354922057604f;

// ------------------------------------------------------------- forward ---

// (largest, sum of 2^(x - largest)) of two sets.
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    if (m == -__builtin_inff()) return float2{m, a.y + b.y};
    return float2{m, a.y * __builtin_amdgcn_exp2f(a.x - m) + b.y * __builtin_amdgcn_exp2f(b.x - m)};
}

// The vocabulary entry that t is, -2 if it is none.
__device__ __forceinline__ int entry_of(int64_t t, int64_t V) { return t >= 0 && t < V ? (int)t : -2; }
// The same of row m's target, -1 if the row is ignored.
__device__ __forceinline__ int target_of(const int64_t* target, int64_t m, int64_t ignore, int64_t V) {
    const int64_t t = target[m];
    return t == ignore ? -1 : entry_of(t, V);
}

// Code i of four.
template <int FMT>
__device__ __forceinline__ float code_value(uint32_t w, int i) {
    const int v = (int)w;
    if constexpr (FMT == 0)
        return i == 0   ? __builtin_amdgcn_cvt_f32_fp8(v, 0)
               : i == 1 ? __builtin_amdgcn_cvt_f32_fp8(v, 1)
               : i == 2 ? __builtin_amdgcn_cvt_f32_fp8(v, 2)
                        : __builtin_amdgcn_cvt_f32_fp8(v, 3);
    else
        return i == 0   ? __builtin_amdgcn_cvt_f32_bf8(v, 0)
               : i == 1 ? __builtin_amdgcn_cvt_f32_bf8(v, 1)
               : i == 2 ? __builtin_amdgcn_cvt_f32_bf8(v, 2)
                        : __builtin_amdgcn_cvt_f32_bf8(v, 3);
}

// sum_k a[k] b[k] of two rows of codes, by a wave.
template <int FA, int FB>
__device__ __forceinline__ float dot_rows(const uint8_t* a, const uint8_t* b, int64_t K) {
    float acc[4] = {};
    for (int64_t k = threadIdx.x % kWaveSize * 16; k < K; k += kWaveSize * 16) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(a + k), y = *reinterpret_cast<const u32x4*>(b + k);
#pragma unroll
        for (int w = 0; w < 4; ++w)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[w] = fmaf(code_value<FA>(x[w], i), code_value<FB>(y[w], i), acc[w]);
    }
    return wave_sum((acc[0] + acc[1]) + (acc[2] + acc[3]));
}

struct LossJoin {
    const float2* part;
    const uint8_t* A;
    const uint8_t* B;
    const float* scale_a;
    const float* scale_b;
    int rowwise;
    const int64_t* target;
    int64_t ignore;
    float* loss;
    float* lse;
    int64_t M, V, K;
    int blocks, group;
};

// Workgroup: `group` rows (a power of two up to 64), 1024 / group slices of their
// column blocks each; a wave for each row's target.
template <int FA, int FB>
__global__ void __launch_bounds__(kLossThreads) loss_kernel(LossJoin p) {
    constexpr int kWaves = kLossThreads / kWaveSize;
    __shared__ float2 s_part[kWaves][64];
    __shared__ float s_target[64];        // logits times log2(e)
    const int64_t M = p.M;
    const int blocks = p.blocks, group = p.group, slices = kLossThreads / group;
    const int wave = threadIdx.x / kWaveSize, lane = threadIdx.x % kWaveSize;
    const int r = threadIdx.x % group;
    const int64_t m = (int64_t)blockIdx.x * group + r;
    float2 v[8];
    auto fetch = [&](int q0) __attribute__((always_inline)) {   // together: one memory latency
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int q = q0 + slices * k;
            v[k] = m < M && q < blocks ? p.part[(int64_t)q * M + m] : float2{-__builtin_inff(), 0.f};
        }
    };
    int q0 = threadIdx.x / group;
    fetch(q0);   // under way while the targets' logits are made
    for (int i = wave; i < group; i += kWaves) {
        const int64_t row = (int64_t)blockIdx.x * group + i;
        if (row >= M) break;
        const int t = entry_of(p.target[row], p.V);   // (of an ignored row too: lse has it)
        if (t < 0) continue;
        const float dot = dot_rows<FA, FB>(p.A + row * p.K, p.B + t * p.K, p.K);
        const float s = (p.rowwise ? p.scale_a[row] : p.scale_a[0]) * kLog2E * (p.rowwise ? p.scale_b[t] : p.scale_b[0]);
        if (lane == 0) s_target[i] = dot * s;
    }
    float2 acc{-__builtin_inff(), 0.f};
    while (true) {
#pragma unroll
        for (int k = 0; k < 8; ++k) acc = merge(acc, v[k]);
        q0 += slices * 8;
        if (q0 - threadIdx.x / group >= blocks) break;
        fetch(q0);
    }
    for (int d = kWaveSize / 2; d >= group; d /= 2)   // a wave's slices of a row
        acc = merge(acc, float2{__shfl_xor(acc.x, d), __shfl_xor(acc.y, d)});
    if (lane < group) s_part[wave][lane] = acc;
    __syncthreads();
    if (threadIdx.x >= group || m >= M) return;
#pragma unroll
    for (int w = 1; w < kWaves; ++w) acc = merge(acc, s_part[w][r]);
    constexpr float kLn2 = 0.69314718055994531f;
    const float others = (acc.x + log2f(acc.y)) * kLn2;       // (all, where there is no target)
    const int64_t target = p.target[m];
    float loss = __builtin_nanf(""), lse = others;
    if (entry_of(target, p.V) >= 0) {
        const float z = s_target[r];
        if (z == -__builtin_inff()) {
            loss = others - z;   // (of no numbers, and where all are -inf, none)
        } else {
            // loss = log(1 + S 2^d), d the others' largest above the target's; lse from the
            // larger of the two, so that nothing cancels.
            const float d = acc.x - z;
            const float rest = d > 0.f ? logf(acc.y + __builtin_amdgcn_exp2f(-d))
                                       : log1pf(acc.y * __builtin_amdgcn_exp2f(d));
            loss = d > 0.f ? fmaf(d, kLn2, rest) : rest;
            lse = fmaf(d > 0.f ? acc.x : z, kLn2, rest);
            if (z == __builtin_inff()) loss = lse = __builtin_nanf("");
        }
    }
    p.loss[m] = target == p.ignore ? 0.f : loss;
    p.lse[m] = lse;
}

__global__ void __launch_bounds__(256) clear_kernel(uint32_t* p, int64_t n) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = 0u;
}

// ------------------------------------------------------------ gradient ---

// What the gradient needs of each row, made once: in x's first pass where dw is asked
// for, else in a kernel of its own.
struct LossGrad {
    static constexpr bool kGiven = true;
    const float* dloss;
    int64_t dloss_stride;
    const int64_t* target;
    int64_t ignore;
    const float* loss;
    const float* lse;
    int64_t M, V;
    float2* rows;          // for the codes' epilogue (LossParams::rows)
    float* factor;         // r
    float* row_scale;      // r / 57344
    float* ones;           // num_ones of 1
    int64_t num_ones;
    uint32_t* counters;    // of the products, cleared
    int num_counters;

    __device__ __forceinline__ void begin() const {
        const int64_t i0 = blockIdx.x * (int64_t)blockDim.x + threadIdx.x, step = (int64_t)gridDim.x * blockDim.x;
        for (int64_t i = i0; i < num_counters; i += step) counters[i] = 0u;
        for (int64_t i = i0; i < num_ones; i += step) ones[i] = 1.f;
    }
    __device__ __forceinline__ float of(int64_t m, bool write) const {
        const int t = target_of(target, m, ignore, V);
        const float l = loss[m], e = lse[m], d = dloss[m * dloss_stride];
        float f = -__builtin_inff(), r = 0.f;
        if (t != -1 && d != 0.f) {
            const float h = l <= 0.f ? 0.f : -expm1f(-l);
            r = d * h;
            if (t < 0 || !(fabsf(e) < __builtin_inff())) r = __builtin_nanf("");
            else if (write && h > 0.f) f = __builtin_fmaf(e, -kLog2E, kLog2E5m2Max - log2f(h));   // (57344 / h may pass the largest float)
        }
        if (write) {
            rows[m] = float2{f, __int_as_float(t)};
            factor[m] = r;
            row_scale[m] = r / kE5m2Max;
        }
        return r;
    }
};

__global__ void __launch_bounds__(256) loss_rows_kernel(LossGrad p) {
    p.begin();
    const int64_t step = gridDim.x * 256ll;
    for (int64_t m = blockIdx.x * 256ll + threadIdx.x; m < p.M; m += step) p.of(m, true);
}

__global__ void __launch_bounds__(256) zero_bf16_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) p[i] = 0;
}

// ---------------------------------------------------------------- host ---

int64_t align256(int64_t n) { return code_up(n, 256) * 256; }
bool at(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int64_t kMaxDim = int64_t(1) << 23;
constexpr int64_t kCounterArea = int64_t(256) << 10;   // the multiply's arrival counters
constexpr int64_t kCodeBytes = int64_t(512) << 20;     // of a piece's codes, both layouts, up to 2^20 rows

int loss_shape(int64_t M, int64_t V, int64_t K) {
    if (M < 0 || M > kMaxDim || V < 1 || V > kMaxDim || K < 16 || K > kMaxDim || K % 16 != 0) return FP8MM_ERR_SHAPE;
    if (M > 0 && !fp8mm::loss_plan_fits(M, V, fp8mm::loss_plan(M, V, K))) return FP8MM_ERR_SHAPE;
    return code_grid_ok(M, K) ? FP8MM_OK : FP8MM_ERR_SHAPE;
}

int loss_operands(const void* A, int fa, const void* B, int fb, const float* sa, const float* sb,
                  const int64_t* target, int mode, int64_t M) {
    if (mode != FP8MM_PER_TENSOR && mode != FP8MM_ROWWISE) return FP8MM_ERR_MODE;
    if ((fa != FP8MM_E4M3FN && fa != FP8MM_E5M2) || (fb != FP8MM_E4M3FN && fb != FP8MM_E5M2)) return FP8MM_ERR_FORMAT;
    if (M > 0 && (!A || !B || !sa || !sb || !target)) return FP8MM_ERR_NULL;
    if (!at(A, 16) || !at(B, 16) || !at(sa, 4) || !at(sb, 4) || !at(target, 8)) return FP8MM_ERR_ALIGN;
    return FP8MM_OK;
}

// A product's launches over the vocabulary (or a piece of it): one, or a second one for
// what would leave most of a round idle.
struct Ranges {
    int64_t end[2];
    int count;
};
Ranges ranges_of(int64_t fixed, int64_t n, int64_t k, bool ping_pong) {
    const int64_t cut = ping_pong ? fp8mm::whole_rounds(fixed, n, k) : n;
    return cut < n ? Ranges{{cut, n}, 2} : Ranges{{n, n}, 1};
}
// (the plan of the whole may be another kernel's)
Ranges logit_ranges(int64_t M, int64_t n, int64_t K) {
    const fp8mm::LossPlan p = fp8mm::loss_plan(M, n, K);
    return ranges_of(M, n, K, p.cfg == fp8mm::ping_pong_config() && p.splits == 1);
}
// dw's rows: those of the codes qt.
Ranges dw_ranges(int64_t n, int64_t K, int64_t Mp) {
    return ranges_of(K, n, Mp,
                     fp8_scaled_mm_select_config(n, K, Mp, FP8MM_ROWWISE, 0, 1) == fp8mm::ping_pong_config() &&
                         fp8_scaled_mm_select_splits(n, K, Mp, FP8MM_ROWWISE, 0, -1) == 1);
}

struct LossSpace {
    int64_t part, total;   // byte offsets (the multiply's workspace is first)
    Ranges ranges;
    fp8mm::LossPlan plan[2];
    int64_t blocks[2];
};

LossSpace loss_space(int64_t M, int64_t V, int64_t K) {
    LossSpace s{};
    if (M == 0) return s;
    s.ranges = logit_ranges(M, V, K);
    int64_t at = 0, mm = 0, blocks = 0;
    for (int i = 0; i < s.ranges.count; ++i) {
        const int64_t n = s.ranges.end[i] - at;
        s.plan[i] = fp8mm::loss_plan(M, n, K);
        s.blocks[i] = fp8mm::loss_blocks(n, s.plan[i]);
        blocks += s.blocks[i];
        mm = std::max(mm, fp8mm::loss_workspace(M, n, s.plan[i]));
        at = s.ranges.end[i];
    }
    s.part = align256(mm);
    s.total = s.part + align256(8 * M * blocks);
    return s;
}

struct GradSpace {
    int64_t mm, rows, factor, row_scale, ones, col_scale, partials, q, qt, qx, sums, total;   // byte offsets
    int64_t piece, ldq, Mp;
    bool one;              // the whole vocabulary in one piece
    int counters;          // to clear (a product leaves those that it uses at zero)
    int dx_splits;         // units of a tile of its dx, 0: the automatic plan
    fp8mm::PairPlan pair;
    CodeJob x;
};

// The two products of the only piece (sizes only).
void products(int64_t M, int64_t V, int64_t K, int64_t ldq, int64_t Mp, fp8mm::Product (&q)[2]) {
    q[0] = fp8mm::Product{nullptr, nullptr, nullptr, nullptr, nullptr, M, K, ldq};
    q[1] = fp8mm::Product{nullptr, nullptr, nullptr, nullptr, nullptr, V, K, Mp};
}

GradSpace grad_space(int64_t M, int64_t V, int64_t K, bool want_dx, bool want_dw) {
    GradSpace g{};
    g.pair.cfg = -1;
    if (M == 0) return g;
    g.Mp = M > 256 ? code_up(M, 64) * 64 : code_up(M, 16) * 16;
    g.piece = kCodeBytes / (2 * g.Mp) / 256 * 256;
    if (g.piece < 256) g.piece = 256;
    g.one = g.piece >= V;
    if (g.one) g.piece = V;
    else g.piece = code_up(code_up(V, code_up(V, g.piece)), 256) * 256;   // (pieces of about one size)
    g.ldq = code_up(g.piece, 16) * 16;
    const int64_t last = g.one ? g.piece : V - (V - 1) / g.piece * g.piece;
    int64_t mm = kCounterArea;
    auto room = [&](int64_t n) { mm = std::max(mm, n); };
    auto product = [&](int64_t m, int64_t n, int64_t k) {
        room(fp8_scaled_mm_workspace_size(m, n, k, FP8MM_ROWWISE, 0, -1, 0));
        g.counters = std::max(g.counters, fp8mm::product_counters({nullptr, nullptr, nullptr, nullptr, nullptr, m, n, k}));
    };
    // The tiles write the codes' zeros past M as far as they reach.
    bool reach = true;
    for (const int64_t n : {g.piece, last}) {
        const Ranges r = logit_ranges(M, n, K);
        for (int i = 0; i < r.count; ++i) {
            const int64_t part = r.end[i] - (i ? r.end[0] : 0);
            const fp8mm::LossPlan plan = fp8mm::loss_plan(M, part, K);
            reach = reach && fp8mm::loss_rows(M, plan) >= g.Mp;
            room(fp8mm::loss_workspace(M, part, plan));
            g.counters = std::max(g.counters, fp8mm::loss_counters(M, part, plan));
        }
    }
    if (!reach) g.Mp = code_up(M, 16) * 16;
    if (want_dx && g.one) {
        g.dx_splits = fp8mm::long_sum_splits(M, K, g.ldq);
        if (g.dx_splits == 0) product(M, K, g.ldq);
    }
    if (want_dw)
        for (const int64_t n : {g.piece, last}) {
            const Ranges r = dw_ranges(n, K, g.Mp);
            for (int i = 0; i < r.count; ++i) product(r.end[i] - (i ? r.end[0] : 0), K, g.Mp);
        }
    if (want_dx && want_dw && g.one && g.dx_splits == 0) {
        fp8mm::Product q[2];
        products(M, V, K, g.ldq, g.Mp, q);
        g.pair = fp8mm::plan_pair(q);
        if (g.pair.cfg >= 0) {
            room(fp8mm::pair_workspace(q, g.pair));
            g.counters = std::max(g.counters, fp8mm::pair_counters(q, g.pair));
        }
    }
    CodeJob& x = g.x;
    x.M = M;
    x.K = K;
    x.Mp = g.Mp;
    x.col_unit = kE5m2Max;
    plan_codes(x);
    g.rows = align256(mm);
    g.factor = g.rows + align256(8 * M);
    g.row_scale = g.factor + align256(4 * M);
    g.ones = g.row_scale + align256(4 * M);
    g.col_scale = g.ones + (want_dw ? align256(4 * g.piece) : 0);
    g.partials = g.col_scale + (want_dw ? align256(4 * K) : 0);
    g.q = g.partials + (want_dw ? align256(code_partials(x, false)) : 0);
    g.qt = g.q + (want_dx ? align256(M * g.ldq) : 0);
    g.qx = g.qt + (want_dw ? align256(g.piece * g.Mp) : 0);
    g.sums = g.qx + (want_dw ? align256(K * g.Mp) : 0);
    g.total = g.sums + (want_dx && (!g.one || g.dx_splits > 0) ? align256(fp8mm::sum_workspace(M, K, g.one ? g.dx_splits : 1)) : 0);
    return g;
}

}  // namespace

extern "C" {

int64_t fp8_linear_cross_entropy_workspace_size(int64_t M, int64_t V, int64_t K) {
    return loss_shape(M, V, K) != FP8MM_OK ? -1 : loss_space(M, V, K).total;
}

int fp8_linear_cross_entropy(const void* A, int a_format, const void* B, int b_format, const float* scale_a,
                             const float* scale_b, const int64_t* target, int64_t ignore_index, float* loss,
                             float* lse, int64_t M, int64_t V, int64_t K, int mode, struct ihipStream_t* stream,
                             void* workspace, int64_t workspace_bytes) {
    int st = loss_shape(M, V, K);
    if (st == FP8MM_OK) st = loss_operands(A, a_format, B, b_format, scale_a, scale_b, target, mode, M);
    if (st != FP8MM_OK) return st;
    if (M == 0) return FP8MM_OK;
    if (!loss || !lse) return FP8MM_ERR_NULL;
    if (!at(loss, 4) || !at(lse, 4) || !at(workspace, 256)) return FP8MM_ERR_ALIGN;
    const LossSpace s = loss_space(M, V, K);
    if (!workspace || workspace_bytes < s.total) return FP8MM_ERR_WORKSPACE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    std::lock_guard<std::mutex> together(fp8mm::enqueue_lock(workspace));
    char* ws = static_cast<char*>(workspace);
    (void)hipGetLastError();
    int counters = 0;
    for (int i = 0; i < s.ranges.count; ++i)
        counters = std::max(counters, fp8mm::loss_counters(M, s.ranges.end[i] - (i ? s.ranges.end[0] : 0), s.plan[i]));
    if (counters > 0)
        hipLaunchKernelGGL(clear_kernel, dim3((unsigned)((counters + 255) / 256)), dim3(256), 0, hs,
                           reinterpret_cast<uint32_t*>(ws), (int64_t)counters);
    float2* part = reinterpret_cast<float2*>(ws + s.part);
    int64_t v0 = 0, blocks = 0;
    for (int i = 0; i < s.ranges.count; ++i) {
        const fp8mm::Logits z{A, a_format, static_cast<const uint8_t*>(B) + v0 * K, b_format, scale_a,
                              mode == FP8MM_ROWWISE ? scale_b + v0 : scale_b, M, s.ranges.end[i] - v0, K, mode};
        st = fp8mm::run_stats(z, s.plan[i], target, part + blocks * M, v0, hs, ws);
        if (st != FP8MM_OK) return st;
        blocks += s.blocks[i];
        v0 = s.ranges.end[i];
    }
    // Rows of a workgroup: whole lines of a column block's rows are better read together, many
    // workgroups better than few (us of the call with groups from 1, 8 and 16 on: 300 x 50000 x 256
    // 29.0, 27.4 and 29.0; 64 x 131072 x 512 48.0, 47.6 and 56.3).
    int group = 1;
    while ((group < 8 && group < M) || (group < 64 && M / group > 256)) group *= 2;
    const LossJoin j{part, static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(B), scale_a, scale_b,
                     mode == FP8MM_ROWWISE, target, ignore_index, loss, lse, M, V, K, (int)blocks, group};
    const dim3 grid((unsigned)code_up(M, group));
    void (*const kernels[2][2])(LossJoin) = {{loss_kernel<0, 0>, loss_kernel<0, 1>}, {loss_kernel<1, 0>, loss_kernel<1, 1>}};
    hipLaunchKernelGGL(kernels[a_format == FP8MM_E5M2][b_format == FP8MM_E5M2], grid, dim3(kLossThreads), 0, hs, j);
    return hipGetLastError() == hipSuccess ? FP8MM_OK : FP8MM_ERR_LAUNCH;
}

int64_t fp8_linear_cross_entropy_backward_workspace_size(int64_t M, int64_t V, int64_t K, int want_dx, int want_dw) {
    return loss_shape(M, V, K) != FP8MM_OK ? -1 : grad_space(M, V, K, want_dx != 0, want_dw != 0).total;
}

int fp8_linear_cross_entropy_backward(const float* dloss, int64_t dloss_stride, const void* A, int a_format,
                                      const void* B, int b_format, const float* scale_a, const float* scale_b,
                                      const int64_t* target, int64_t ignore_index, const float* loss,
                                      const float* lse, const void* x, const void* wt, int wt_format,
                                      const float* wt_scale, void* dx, void* dw, int64_t M, int64_t V, int64_t K,
                                      int mode, struct ihipStream_t* stream, void* workspace,
                                      int64_t workspace_bytes) {
    int st = loss_shape(M, V, K);
    if (st == FP8MM_OK && dloss_stride != 0 && dloss_stride != 1) st = FP8MM_ERR_SHAPE;
    if (st == FP8MM_OK) st = loss_operands(A, a_format, B, b_format, scale_a, scale_b, target, mode, M);
    if (st != FP8MM_OK) return st;
    if (dx && wt_format != FP8MM_E4M3FN && wt_format != FP8MM_E5M2) return FP8MM_ERR_FORMAT;
    if (M > 0 && ((!dx && !dw) || !dloss || !loss || !lse || (dx && (!wt || !wt_scale)) || (dw && !x)))
        return FP8MM_ERR_NULL;
    if (!at(dloss, 4) || !at(loss, 4) || !at(lse, 4) || !at(x, 2) || !at(wt, 16) || !at(wt_scale, 4) || !at(dx, 2) ||
        !at(dw, 2) || !at(workspace, 256))
        return FP8MM_ERR_ALIGN;
    GradSpace g = grad_space(M, V, K, dx != nullptr, dw != nullptr);
    if (M > 0 && (!workspace || workspace_bytes < g.total)) return FP8MM_ERR_WORKSPACE;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return FP8MM_ERR_DEVICE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (M == 0) {
        if (dw)
            hipLaunchKernelGGL(zero_bf16_kernel, dim3(2048), dim3(256), 0, hs, static_cast<uint16_t*>(dw), V * K);
        return hipGetLastError() == hipSuccess ? FP8MM_OK : FP8MM_ERR_LAUNCH;
    }
    std::lock_guard<std::mutex> together(fp8mm::enqueue_lock(workspace));
    char* ws = static_cast<char*>(workspace);
    auto f32 = [&](int64_t offset) { return reinterpret_cast<float*>(ws + offset); };
    uint8_t* q = dx ? reinterpret_cast<uint8_t*>(ws + g.q) : nullptr;
    uint8_t* qt = dw ? reinterpret_cast<uint8_t*>(ws + g.qt) : nullptr;
    LossGrad p{};
    p.dloss = dloss;
    p.dloss_stride = dloss_stride;
    p.target = target;
    p.ignore = ignore_index;
    p.loss = loss;
    p.lse = lse;
    p.M = M;
    p.V = V;
    p.rows = reinterpret_cast<float2*>(ws + g.rows);
    p.factor = f32(g.factor);
    p.row_scale = f32(g.row_scale);
    p.ones = f32(g.ones);
    p.num_ones = dw ? g.piece : 0;
    p.counters = reinterpret_cast<uint32_t*>(ws);
    p.num_counters = g.counters;
    if (dw) {
        CodeJob& c = g.x;
        c.x = x;
        c.factor = p.factor;
        c.col_max = f32(g.partials);
        c.col_scale = f32(g.col_scale);
        c.q_cols = reinterpret_cast<uint8_t*>(ws + g.qx);
        launch_codes<bf16_t, 0, false, false>(c, p, hs);
    } else {
        hipLaunchKernelGGL(loss_rows_kernel, dim3((unsigned)std::min<int64_t>(code_up(M, 256), 256)), dim3(256), 0, hs, p);
    }
    if (hipGetLastError() != hipSuccess) return FP8MM_ERR_LAUNCH;
    const int64_t Vt = code_up(V, 16) * 16;
    for (int64_t v0 = 0; v0 < V; v0 += g.piece) {
        const int64_t n = V - v0 < g.piece ? V - v0 : g.piece;
        const int64_t ldq = code_up(n, 16) * 16;
        const Ranges r = logit_ranges(M, n, K);
        for (int i = 0; i < r.count; ++i) {
            const int64_t c0 = i ? r.end[0] : 0, v = v0 + c0;
            const fp8mm::Logits z{A, a_format, static_cast<const uint8_t*>(B) + v * K, b_format, scale_a,
                                  mode == FP8MM_ROWWISE ? scale_b + v : scale_b, M, r.end[i] - c0, K, mode};
            st = fp8mm::run_codes(z, fp8mm::loss_plan(M, z.V, K), p.rows, q ? q + c0 : nullptr, ldq,
                                  qt ? qt + c0 * g.Mp : nullptr, g.Mp, v, hs, ws);
            if (st != FP8MM_OK) return st;
        }
        uint16_t* dw_piece = static_cast<uint16_t*>(dw) + (dw ? v0 * K : 0);
        if (g.one && dx && dw && wt_format == FP8MM_E4M3FN && g.pair.cfg >= 0) {
            const fp8mm::Product two[2] = {
                {q, wt, p.row_scale, wt_scale, dx, M, K, ldq},
                {qt, ws + g.qx, p.ones, f32(g.col_scale), dw, V, K, g.Mp}};
            return fp8mm::run_pair(two, g.pair, hs, ws);
        }
        // dx first: the caches still hold the codes, and what dw writes would push them out.
        if (dx && g.one && g.dx_splits == 0)
            st = fp8_scaled_mm_typed(q, FP8MM_E5M2, wt, wt_format, p.row_scale, wt_scale, nullptr, dx, M, K, ldq,
                                     FP8MM_ROWWISE, stream, -1, 0, ws, g.rows);
        else if (dx)
            st = fp8mm::run_sum({q, static_cast<const uint8_t*>(wt) + v0, wt_format, p.row_scale, wt_scale, dx, M, K,
                                 ldq, Vt, v0 == 0, v0 + n == V, g.one ? g.dx_splits : 1},
                                hs, ws + g.sums);
        if (st != FP8MM_OK) return st;
        const Ranges d = dw ? dw_ranges(n, K, g.Mp) : Ranges{};
        for (int i = 0; i < d.count; ++i) {
            const int64_t c0 = i ? d.end[0] : 0;
            st = fp8mm::run_streamed({qt + c0 * g.Mp, ws + g.qx, p.ones, f32(g.col_scale), dw_piece + c0 * K,
                                      d.end[i] - c0, K, g.Mp},
                                     hs, ws, g.rows);
            if (st != FP8MM_OK) return st;
        }
        if (st != FP8MM_OK) return st;
    }
    return FP8MM_OK;
}

}  // extern "C"
