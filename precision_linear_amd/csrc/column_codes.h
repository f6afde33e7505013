// Float8 codes of a matrix with one scale for each column, transposed, and, beside
// them, with one scale for each row, in place: the two layouts in which products
// over the columns and over the rows take their operands.
//
// For x (M x K, bf16 or fp32, its rows times factors if given):
//     q_cols[k][m] = RNE(x[m][k] / col_scale[k]),  col_scale[k] = max_m |x| / qmax
//     q_rows[m][k] = RNE(x[m][k] / row_scale[m]),  row_scale[m] = max_k |x| / qmax
// with correctly rounded quotients, as in fp8_quantize.h.  Both need maxima of whole
// rows and columns, so x is read twice (but for column codes of few rows, few_rows_kernel):
//   1. maxima_kernel: partial maxima of columns (by strips of rows) and of rows (by
//      blocks of columns), with the rows' factors made on the way;
//   2. scales_kernel joins them, unless they are so few that pass 3 does it itself;
//   3. codes_kernel.
// A row whose factor is 0 counts as zeros whatever it holds.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "fp8_convert.h"
#include "lane_ops.h"

namespace {

constexpr int kCodeThreads = 256;
constexpr int kCodeCols = 128;                               // of a workgroup: 16 lanes x 8 columns
constexpr int kCodeColLanes = kCodeCols / 8;                 // 16: a DPP row
constexpr int kCodeRowLanes = kCodeThreads / kCodeColLanes;  // 16
constexpr int kCodeUnroll = 4;                               // rows in flight per thread in pass 1
constexpr int kCodeJoin = 64;                                // partial maxima that pass 3 joins itself

// A kernel argument that makes the rows' factors in pass 1: of(m, write) is row m's,
// and where `write` is set leaves it in `factor`; begin() is what else the launch does.
struct NoFactor {
    static constexpr bool kGiven = false;
    __device__ __forceinline__ void begin() const {}
    __device__ __forceinline__ float of(int64_t, bool) const { return 1.f; }
};

struct CodeJob {
    const void* x;
    const float* factor;   // M, for pass 3 where there are factors
    int64_t M, K;
    int64_t Mp;            // row length of q_cols, M rounded up to 16 or more (zeros there)
    int blocks, parts;     // column blocks, strips of rows in pass 1
    int64_t strip;
    float* col_max;        // [parts][K]
    float* row_max;        // [blocks][M], null without row codes
    float* col_scale;      // K
    float* row_scale;      // M
    uint8_t* q_cols;
    uint8_t* q_rows;       // may be null
    // Divides the column scales that are written (the quotients are of the scales
    // as above).
    float col_unit;
};

// 8 elements times the row's factor.
template <class T, bool FACTOR>
__device__ __forceinline__ void code_values(const Raw8<T>& a, float factor, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        f[i] = a.get(i);
        if constexpr (FACTOR) f[i] = factor == 0.f ? 0.f : f[i] * factor;
    }
}

template <class T, class F, bool ROWS, bool NT>
__global__ void __launch_bounds__(kCodeThreads) maxima_kernel(CodeJob p, F factors) {
    constexpr bool FACTOR = F::kGiven;
    __shared__ float s_max[kCodeRowLanes][kCodeCols];
    factors.begin();
    const T* x = static_cast<const T*>(p.x);
    const int cl = threadIdx.x % kCodeColLanes, rl = threadIdx.x / kCodeColLanes;
    const int part = blockIdx.x / p.blocks, cb = blockIdx.x - part * p.blocks;
    const int64_t col = (int64_t)cb * kCodeCols + cl * 8;
    const bool ok = col < p.K;                         // K is a multiple of 16
    const int64_t r1 = min(p.M, (part + 1) * p.strip);
    float cmax[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cmax[i] = 0.f;
    for (int64_t r = part * p.strip + rl; r < r1; r += kCodeRowLanes * kCodeUnroll) {
        Raw8<T> a[kCodeUnroll];
        float factor[kCodeUnroll];
#pragma unroll
        for (int u = 0; u < kCodeUnroll; ++u) {
            const int64_t row = r + u * kCodeRowLanes;
            a[u].zero();
            if (ok && row < r1) a[u].template load<NT>(x + row * p.K + col);
        }
#pragma unroll
        for (int u = 0; u < kCodeUnroll; ++u) {
            const int64_t row = r + u * kCodeRowLanes;
            factor[u] = 1.f;
            if constexpr (FACTOR)
                if (row < r1) factor[u] = factors.of(row, cb == 0 && cl == 0);
        }
#pragma unroll
        for (int u = 0; u < kCodeUnroll; ++u) {
            float f[8], rmax = 0.f;
            code_values<T, FACTOR>(a[u], factor[u], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cmax[i] = fmaxf(cmax[i], fabsf(f[i]));
                if constexpr (ROWS) rmax = fmaxf(rmax, fabsf(f[i]));
            }
            if constexpr (ROWS) {
                const int64_t row = r + u * kCodeRowLanes;
                rmax = row16_max(rmax);
                if (cl == 0 && row < r1) p.row_max[cb * p.M + row] = rmax;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s_max[rl][cl * 8 + i] = cmax[i];
    __syncthreads();
    const int64_t c = (int64_t)cb * kCodeCols + threadIdx.x;
    if (threadIdx.x >= kCodeCols || c >= p.K) return;
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kCodeRowLanes; ++i) m = fmaxf(m, s_max[i][threadIdx.x]);
    p.col_max[part * p.K + c] = m;
}

// The largest of p[0], p[n], ... of `parts` values, every step-th from `first` on, U
// loaded at a time (one memory latency).
template <int U>
__device__ __forceinline__ float join_max(const float* p, int64_t n, int parts, int first, int step) {
    float m = 0.f;
    for (int q0 = first; q0 < parts; q0 += step * U) {
        float v[U];
#pragma unroll
        for (int k = 0; k < U; ++k) v[k] = q0 + step * k < parts ? p[(q0 + step * k) * n] : 0.f;
#pragma unroll
        for (int k = 0; k < U; ++k) m = fmaxf(m, v[k]);
    }
    return m;
}

// Workgroup: 64 rows or columns, 16 slices of their partial maxima each.  The joined
// maxima take the place of the first partial ones of what the workgroup joins.
constexpr int kScaleGroup = 64, kScaleSlices = 16;
__global__ void __launch_bounds__(kScaleGroup* kScaleSlices) scales_kernel(CodeJob p, int blocks_rows) {
    __shared__ float s_max[kScaleSlices][kScaleGroup];
    const int lane = threadIdx.x % kScaleGroup, slice = threadIdx.x / kScaleGroup;
    const bool rows = (int)blockIdx.x < blocks_rows;
    const int64_t n = rows ? p.M : p.K;
    const int64_t i = (int64_t)(rows ? blockIdx.x : blockIdx.x - blocks_rows) * kScaleGroup + lane;
    float* part = rows ? p.row_max : p.col_max;
    s_max[slice][lane] = i < n ? join_max<8>(part + i, n, rows ? p.blocks : p.parts, slice, kScaleSlices) : 0.f;
    __syncthreads();
    if (slice != 0 || i >= n) return;
    float m = 0.f;
#pragma unroll
    for (int q = 0; q < kScaleSlices; ++q) m = fmaxf(m, s_max[q][lane]);
    part[i] = m;
}

// Workgroup: a tile of R rows x 128 columns.  A thread takes 4 consecutive rows of 8
// columns at a time, so that 4 codes of a column make one word of the transposed
// tile in LDS: 128 lines of R / 16 chunks of 16 bytes, chunk c of line n at c ^ ((n
// >> 3) % (R / 16)), which spreads the 16 column lanes over the banks.
template <class T, int FMT, bool FACTOR, bool ROWS, int R, bool NT>
__global__ void __launch_bounds__(kCodeThreads) codes_kernel(CodeJob p, int col_parts, int row_parts) {
    constexpr float kMax = Fp8Fmt<FMT>::kMax;
    constexpr int kChunks = R / 16;
    __shared__ __attribute__((aligned(16))) uint32_t s_t[kCodeCols][R / 4];
    __shared__ float s_col[2][kCodeCols], s_row[3][R];   // scales, reciprocals, factors
    __shared__ int s_slow[kCodeThreads / kWaveSize];
    const T* x = static_cast<const T*>(p.x);
    const int cl = threadIdx.x % kCodeColLanes, rl = threadIdx.x / kCodeColLanes;
    // Last strips first: the caches still hold them from pass 1.
    const int64_t turn = blockIdx.x / p.blocks;
    const int cb = (int)(blockIdx.x - turn * p.blocks);
    const int64_t strip = gridDim.x / p.blocks - 1 - turn;
    const int64_t col = (int64_t)cb * kCodeCols + cl * 8, row0 = strip * R;
    const bool ok = col < p.K;
    constexpr int kSteps = R / (4 * kCodeRowLanes);
    Raw8<T> a[4];
    auto fetch = [&](int it) __attribute__((always_inline)) {
        const int64_t r = row0 + (it * kCodeRowLanes + rl) * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[k].zero();
            if (ok && r + k < p.M) a[k].template load<NT>(x + (r + k) * p.K + col);
        }
    };
    fetch(0);   // under way while the scales are found
    static_assert(kCodeThreads >= kCodeCols + R, "one thread for each row and column");
    int slow = 0;   // whether a division here is outside the fast one's range
    {
        const int t = threadIdx.x;
        if (t < kCodeCols) {
            const int64_t c = (int64_t)cb * kCodeCols + t;
            float s = 0.f;
            if (c < p.K) {
                s = join_max<32>(p.col_max + c, p.K, col_parts, 0, 1) / kMax;
                if (strip == 0) p.col_scale[c] = s / p.col_unit;
            }
            const Div d = make_div(s);
            slow = !d.fast && s != 0.f;
            s_col[0][t] = s;
            s_col[1][t] = s == 0.f ? 0.f : d.r;
        } else if (t < kCodeCols + R) {
            const int64_t r = row0 + t - kCodeCols;
            float s = 0.f, factor = 1.f;
            if (r < p.M) {
                if constexpr (ROWS) {
                    s = join_max<32>(p.row_max + r, p.M, row_parts, 0, 1) / kMax;
                    if (cb == 0) p.row_scale[r] = s;
                }
                if constexpr (FACTOR) factor = p.factor[r];
            }
            const Div d = make_div(s);
            slow = !d.fast && s != 0.f;
            s_row[0][t - kCodeCols] = s;
            s_row[1][t - kCodeCols] = s == 0.f ? 0.f : d.r;
            s_row[2][t - kCodeCols] = factor;
        }
        const bool any = __ballot(slow) != 0;
        if (t % kWaveSize == 0) s_slow[t / kWaveSize] = any;
        __syncthreads();
        static_assert(kCodeThreads / kWaveSize == 4, "four waves' flags");
        slow = __builtin_amdgcn_readfirstlane(s_slow[0] | s_slow[1] | s_slow[2] | s_slow[3]);
    }
    float cs[8], cr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = s_col[0][cl * 8 + i];
        cr[i] = s_col[1][cl * 8 + i];
    }
    // The 4 rows of group `mg` in f, FAST: every division here is in the fast one's range.
    auto rows_of = [&](auto fast, int mg, const float (&f)[4][8]) __attribute__((always_inline)) {
        constexpr bool FAST = decltype(fast)::value;
        const int64_t r = row0 + mg * 4;
        // value / s: with s = 0 every finite value gives 0.
        auto over = [](float v, float s, float rr) __attribute__((always_inline)) {
            const Div d{s, rr, true};
            if constexpr (FAST) return quant1<FMT, true>(v, d);
            else return s == 0.f ? v * 0.f : quant1<FMT, false>(v, d);
        };
        if constexpr (ROWS) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float s = s_row[0][mg * 4 + k], rr = s_row[1][mg * 4 + k];
                u32x2 codes;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int w = Fp8Fmt<FMT>::template cvt_pk<false>(over(f[k][4 * h], s, rr), over(f[k][4 * h + 1], s, rr), 0);
                    codes[h] = (uint32_t)Fp8Fmt<FMT>::template cvt_pk<true>(over(f[k][4 * h + 2], s, rr),
                                                                            over(f[k][4 * h + 3], s, rr), w);
                }
                if (ok && r + k < p.M) store_hinted<NT>(reinterpret_cast<u32x2*>(p.q_rows + (r + k) * p.K + col), codes);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int w = Fp8Fmt<FMT>::template cvt_pk<false>(over(f[0][i], cs[i], cr[i]), over(f[1][i], cs[i], cr[i]), 0);
            s_t[cl * 8 + i][(((mg >> 2) ^ (cl % kChunks)) << 2) | (mg & 3)] =
                (uint32_t)Fp8Fmt<FMT>::template cvt_pk<true>(over(f[2][i], cs[i], cr[i]), over(f[3][i], cs[i], cr[i]), w);
        }
    };
#pragma unroll 1
    for (int it = 0; it < kSteps; ++it) {
        const int mg = it * kCodeRowLanes + rl;            // group of 4 rows in the tile
        float f[4][8];
#pragma unroll
        for (int k = 0; k < 4; ++k) code_values<T, FACTOR>(a[k], s_row[2][mg * 4 + k], f[k]);
        if (it + 1 < kSteps) fetch(it + 1);
        if (!slow) rows_of(std::true_type(), mg, f);
        else rows_of(std::false_type(), mg, f);
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kCodeCols * kChunks / kCodeThreads; ++it) {
        const int q = it * kCodeThreads + threadIdx.x;
        const int n = q / kChunks, c = q % kChunks;
        const int64_t line = (int64_t)cb * kCodeCols + n, m = row0 + c * 16;
        if (line < p.K && m < p.Mp)
            *reinterpret_cast<u32x4*>(p.q_cols + line * p.Mp + m) =
                *reinterpret_cast<const u32x4*>(&s_t[n][(c ^ ((n >> 3) % kChunks)) << 2]);
    }
}

// Column codes of up to 2 THREADS rows in one launch: a workgroup holds 16 columns of them
// all in its registers, 8 columns a lane of rows 4 r .. 4 r + 3 for r = threadIdx.x / 2, so x
// is read once and nothing is left to join.  (us of the cross entropy's gradient on one
// MI355X with the two passes and with this: 100 x 32000 x 1024 57.3 and 52.6, 1001 x 50255 x
// 2048 349.7 and 345.8; 5.1 and 12.5 of them here, memory latencies one after the other.)
constexpr int kFewCols = 16, kFewLanes = kFewCols / 8;
// Over the lanes of a wave with the same lane % kFewLanes.
__device__ __forceinline__ float few_max(float x) {
    static_assert(kFewLanes == 2, "the first step is lane ^ 2");
    constexpr int kTurn4 = 0x124, kTurn8 = 0x128;   // of 16 lanes
    x = fmaxf(x, dpp<kSwap2>(x));
    x = fmaxf(x, dpp<kTurn4>(x));
    x = fmaxf(x, dpp<kTurn8>(x));
    uint32_t h = __float_as_uint(x);
    const auto half = __builtin_amdgcn_permlane32_swap(h, h, false, false);
    x = fmaxf(__uint_as_float(half[0]), __uint_as_float(half[1]));
    h = __float_as_uint(x);
    const auto row = __builtin_amdgcn_permlane16_swap(h, h, false, false);
    return fmaxf(__uint_as_float(row[0]), __uint_as_float(row[1]));
}
// Row codes are made by further workgroups, a wave a row, which read x once more (us a call
// from Python with the two passes and with this: 3 x 112 and 100 x 4096 fp32 13.2 and
// 10.1, 128 x 8192 13.2 and 10.1, 1024 x 1024 13.3 and 10.1, but 1000 x 4160 bf16 13.1 and 13.1, 32 x 28672
// 16.2 and 17.9, 1024 x 8192 17.2 and 23.5).
constexpr int64_t kFewElements = int64_t(1) << 20, kFewRowLength = 8192;
template <class T, int FMT>
__device__ __forceinline__ void row_codes(const CodeJob& p, int64_t row) {
    constexpr int kAhead = 4, kStep = kWaveSize * 8;   // elements of a wave's load; loads in flight
    const T* x = static_cast<const T*>(p.x) + row * p.K;
    const int64_t first = threadIdx.x % kWaveSize * 8;
    Raw8<T> a[kAhead];
    auto fetch = [&](int64_t c0) __attribute__((always_inline)) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            a[k].zero();
            if (c0 + k * kStep < p.K) a[k].load(x + c0 + k * kStep);
        }
    };
    float m = 0.f;
    for (int64_t c0 = first; c0 < p.K; c0 += kAhead * kStep) {
        fetch(c0);
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(a[k].get(i)));
    }
    const float s = wave_max(m) / Fp8Fmt<FMT>::kMax;
    if (threadIdx.x % kWaveSize == 0) p.row_scale[row] = s;
    const Div d = make_div(s);
    const bool fast = d.fast;
    for (int64_t c0 = first; c0 < p.K; c0 += kAhead * kStep) {
        if (p.K > kAhead * kStep) fetch(c0);   // (else a still holds the row)
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            float y[8];
            if (fast) {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = quant1<FMT, true>(a[k].get(i), d);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = s == 0.f ? a[k].get(i) * 0.f : quant1<FMT, false>(a[k].get(i), d);
            }
            u32x2 codes;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int w = Fp8Fmt<FMT>::template cvt_pk<false>(y[4 * h], y[4 * h + 1], 0);
                codes[h] = (uint32_t)Fp8Fmt<FMT>::template cvt_pk<true>(y[4 * h + 2], y[4 * h + 3], w);
            }
            const int64_t c = c0 + k * kStep;
            if (c < p.K) *reinterpret_cast<u32x2*>(p.q_rows + row * p.K + c) = codes;
        }
    }
}
template <class T, int FMT, class F, bool ROWS, int THREADS>
__global__ void __launch_bounds__(THREADS) few_rows_kernel(CodeJob p, F factors) {
    constexpr int kWaves = THREADS / kWaveSize;
    if constexpr (ROWS) {
        const int64_t block = (int64_t)blockIdx.x - p.K / kFewCols;
        if (block >= 0) {
            const int64_t row = block * kWaves + threadIdx.x / kWaveSize;
            if (row < p.M) row_codes<T, FMT>(p, row);
            return;
        }
    }
    __shared__ float s_factor[2 * THREADS];
    __shared__ float s_max[kWaves][kFewCols], s_col[2][kFewCols];
    __shared__ int s_slow;
    const T* x = static_cast<const T*>(p.x);
    const int cl = threadIdx.x % kFewLanes, r = threadIdx.x / kFewLanes * 4;
    const int64_t col0 = (int64_t)blockIdx.x * kFewCols, col = col0 + cl * 8;   // K is a multiple of 16
    Raw8<T> a[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        a[k].zero();
        if (r + k < p.M) a[k].load(x + (r + k) * p.K + col);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int i = k * THREADS + threadIdx.x;
        s_factor[i] = i < p.M ? factors.of(i, blockIdx.x == 0) : 1.f;
    }
    factors.begin();
    __syncthreads();
    float f[4][8], cs[8], cr[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) code_values<T, F::kGiven>(a[k], s_factor[r + k], f[k]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float m = 0.f;   // (no NaN)
#pragma unroll
        for (int k = 0; k < 4; ++k) m = fmaxf(m, fabsf(f[k][i]));
        m = few_max(m);
        if (threadIdx.x % kWaveSize < kFewLanes) s_max[threadIdx.x / kWaveSize][cl * 8 + i] = m;
    }
    __syncthreads();
    if (threadIdx.x < kWaveSize) {
        bool slow = false;   // whether a division here is outside the fast one's range
        if (threadIdx.x < kFewCols) {
            float m = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) m = fmaxf(m, s_max[w][threadIdx.x]);
            const float s = m / Fp8Fmt<FMT>::kMax;
            p.col_scale[col0 + threadIdx.x] = s / p.col_unit;
            const Div d = make_div(s);
            slow = !d.fast && s != 0.f;
            s_col[0][threadIdx.x] = s;
            s_col[1][threadIdx.x] = s == 0.f ? 0.f : d.r;
        }
        slow = __any(slow);
        if (threadIdx.x == 0) s_slow = slow;
    }
    __syncthreads();
    const bool slow = __builtin_amdgcn_readfirstlane(s_slow);
    if (r >= p.Mp) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = s_col[0][cl * 8 + i];
        cr[i] = s_col[1][cl * 8 + i];
    }
    auto codes = [&](auto fast) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float y[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const Div d{cs[i], cr[i], true};
                if constexpr (decltype(fast)::value) y[k] = quant1<FMT, true>(f[k][i], d);
                else y[k] = cs[i] == 0.f ? f[k][i] * 0.f : quant1<FMT, false>(f[k][i], d);
            }
            const int w = Fp8Fmt<FMT>::template cvt_pk<false>(y[0], y[1], 0);
            *reinterpret_cast<int*>(p.q_cols + (col + i) * p.Mp + r) = Fp8Fmt<FMT>::template cvt_pk<true>(y[2], y[3], w);
        }
    };
    if (!slow) codes(std::true_type());
    else codes(std::false_type());
}

// ---------------------------------------------------------------- host ---

inline int64_t code_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Blocks, strips and the number of partial maxima, from the sizes.
inline void plan_codes(CodeJob& p) {
    p.blocks = (int)code_up(p.K, kCodeCols);
    const int64_t round = kCodeRowLanes * kCodeUnroll;
    p.strip = round;
    while (p.strip < 256 && code_up(p.M, 2 * p.strip) * p.blocks >= 2048) p.strip *= 2;
    if (code_up(p.M, p.strip) > kCodeJoin && p.M <= 65536)
        p.strip = code_up(code_up(p.M, kCodeJoin), round) * round;
    p.parts = (int)code_up(p.M, p.strip);
}
// Bytes of partial maxima: col_max, then row_max.
inline int64_t code_partials(const CodeJob& p, bool rows) {
    return 4 * ((int64_t)p.parts * p.K + (rows ? (int64_t)p.blocks * p.M : 0));
}
// Whether the launches' threads, of which there are fewer than 2^32, can be counted (pass 1
// takes strips of 128 rows or more, but for a few thousand workgroups).
inline bool code_grid_ok(int64_t M, int64_t K) {
    return code_up(M, 128) * code_up(K, kCodeCols) * kCodeThreads <= UINT32_MAX &&
           (code_up(M, kScaleGroup) + code_up(K, kScaleGroup)) * kScaleGroup * kScaleSlices <= UINT32_MAX;
}

template <class T, int FMT, bool ROWS, bool NT, class F>
void launch_codes(const CodeJob& p, const F& factors, hipStream_t hs) {
    constexpr bool FACTOR = F::kGiven;
    if constexpr (!NT) {
        const int threads = p.Mp <= 256 ? 128 : 512;
        const dim3 grid((unsigned)(p.K / kFewCols + (ROWS ? code_up(p.M, threads / kWaveSize) : 0)));
        if (p.Mp <= 1024 && (!ROWS || (p.K <= kFewRowLength && p.M * p.K <= kFewElements))) {
            if (threads == 128) hipLaunchKernelGGL((few_rows_kernel<T, FMT, F, ROWS, 128>), grid, dim3(128), 0, hs, p, factors);
            else hipLaunchKernelGGL((few_rows_kernel<T, FMT, F, ROWS, 512>), grid, dim3(512), 0, hs, p, factors);
            return;
        }
    }
    hipLaunchKernelGGL((maxima_kernel<T, F, ROWS, NT>), dim3((unsigned)((int64_t)p.parts * p.blocks)),
                       dim3(kCodeThreads), 0, hs, p, factors);
    int col_parts = p.parts, row_parts = p.blocks;
    if (col_parts > kCodeJoin || (ROWS && row_parts > kCodeJoin)) {
        const int rows = ROWS ? (int)code_up(p.M, kScaleGroup) : 0, cols = (int)code_up(p.K, kScaleGroup);
        hipLaunchKernelGGL(scales_kernel, dim3((unsigned)(rows + cols)), dim3(kScaleGroup * kScaleSlices), 0, hs, p, rows);
        col_parts = row_parts = 1;
    }
    // 64 rows a workgroup (half the work) where the grid is small.
    if (code_up(p.M, 128) * p.blocks >= 512)
        hipLaunchKernelGGL((codes_kernel<T, FMT, FACTOR, ROWS, 128, NT>), dim3((unsigned)(code_up(p.M, 128) * p.blocks)),
                           dim3(kCodeThreads), 0, hs, p, col_parts, row_parts);
    else
        hipLaunchKernelGGL((codes_kernel<T, FMT, FACTOR, ROWS, 64, NT>), dim3((unsigned)(code_up(p.M, 64) * p.blocks)),
                           dim3(kCodeThreads), 0, hs, p, col_parts, row_parts);
}

}  // namespace
