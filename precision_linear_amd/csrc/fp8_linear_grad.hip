// The gradient of the FP8 linear layer for gfx950 (MI355X) (formulas:
// include/fp8_linear.h).
//
// dz = dy act'(z) is needed in float8 twice, with one scale for each row (for
// dx) and with one for each column, transposed (for dw, whose products run
// over the rows).  Both scales need the maxima of whole rows and columns, so dz
// is computed twice rather than written out in 32 bits:
//   1. grad_stats_kernel: maxima of dz's rows and columns, sums of its columns
//      (dbias), maxima of x's columns, as partial results; it also clears the
//      products' arrival counters, so that the workspace may hold anything;
//   2. grad_scales_kernel: joins them into the scales and dbias; with few
//      partial results the third pass does that itself;
//   3. grad_quantize_kernel: the codes of dz (row-major, and transposed) and of
//      x (transposed);
//   4. the two products, on the scaled multiply's kernels: in one launch where
//      they fill the GPU better together (small ones), else in two.
// Passes 1 and 3 are bound by memory (where the caches feed them, by arithmetic):
// 2 x 4 bytes read and 2 bytes written for an element of dz, against 4 K operations
// of the products.  4096 x 28672 x 8192 with gelu: 98 + 5 + 142 us of 1542; the
// products run at 2.9 to 3.1 PFLOP/s.
//
// Nothing is summed in an order that depends on timing: sums go through
// partial results joined in a fixed order.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/fp8_linear.h"
#include "activation.h"
#include "enqueue_lock.h"
#include "fp8_convert.h"
#include "fp8_pair.h"
#include "lane_ops.h"

namespace {

constexpr int kThreadsG = 256;
constexpr int kTileCols = 128;                      // 16 lanes x 8 columns
constexpr int kColLanes = kTileCols / 8;            // 16: a DPP row
constexpr int kRowLanes = kThreadsG / kColLanes;    // 16
constexpr int kTileRows = 128;                      // of the quantisation's tiles (64 in small grids)
constexpr int kStatUnroll = 4;                      // rows in flight per thread

struct Grad {
    const bf16_t* dy;
    const bf16_t* z;       // null for kActNone
    const bf16_t* x;       // null without dw
    int64_t M, N, K;
    int64_t Mp;            // row length of the transposed codes: M rounded up to 16, or to 64
                           // (whole write segments of pass 3) where that is little
    int blocks_n, blocks_k;   // column blocks of dz and x (0 without dw)
    int parts;             // row strips of pass 1
    int64_t strip;         // rows of a strip
    int want_rows, want_cols;   // dz codes by rows (dx), by columns (dw)
    // Partial results: [blocks_n][M], [parts][N], [parts][N], [parts][K]
    float* row_max;
    float* col_max;
    float* col_sum;
    float* x_max;
    // Scales, and their reciprocals right behind them: 2 M, 2 N, 2 K
    float* row_scale;
    float* col_scale;
    float* x_scale;
    float* dbias;          // may be null
    uint8_t* q_rows;       // M x N
    uint8_t* q_cols;       // N x Mp
    uint8_t* q_x;          // K x Mp
    uint32_t* counters;    // of the products
    int num_counters;
};

// dz of 8 elements.
template <int ACT>
__device__ __forceinline__ void dz8(const Raw8<bf16_t>& dy, const Raw8<bf16_t>& z, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = dy.get(i) * slope<ACT>(z.get(i));
}

// The gelus' slopes from a table in LDS.  z has 16 bits, and the slope of z is 1
// less that of -z, so the 1664 values of slope(-t) for 2^-9 <= t < 16 are all there
// is: below, it is 1/2 - sqrt(2 / pi) t (within 5e-9), above, 0 (in fp32).  The
// small side is the one that is kept: far below 0 the slope has slope()'s own
// relative accuracy, above 0 one rounding more.  About 13 instructions for some 30,
// which the passes are bound by where the caches feed them (the whole gradient on
// one MI355X, gelu, us without and with: 4069 x 12720 x 176 174 and 167, 8192 x 4096
// x 1024 155 and 148, 4096 x 28672 x 8192 1538 and 1513; under 512 tiles of dz the
// table's filling costs more, 1024 x 2048 x 8192 62 and 64).
template <int ACT> constexpr bool kHasTable = ACT == kActGelu || ACT == kActGeluTanh;
constexpr uint32_t kTableFirst = 0x3b00, kTableEnd = 0x4180;   // bf16 2^-9 and 16
constexpr int kTableSize = (int)(kTableEnd - kTableFirst);

template <int ACT>
__device__ __forceinline__ void fill_table(float* table) {
    for (int i = threadIdx.x; i < kTableSize; i += kThreadsG)
        table[i] = slope<ACT>(-__uint_as_float((kTableFirst + (uint32_t)i) << 16));
}

__device__ __forceinline__ void dz8_table(const Raw8<bf16_t>& dy, const Raw8<bf16_t>& z, const float* table,
                                          float (&f)[8]) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 most{0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const u16x2 t = __builtin_bit_cast(u16x2, z.v[w] & 0x7fff7fffu);
        most = __builtin_elementwise_max(most, t);
        u16x2 at = __builtin_elementwise_sub_sat(t, u16x2{kTableFirst, kTableFirst});
        at = __builtin_elementwise_min(at, u16x2{kTableSize - 1, kTableSize - 1});
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float v = z.get(2 * w + k);
            const float h = fabsf(v) < 0x1p-9f ? fmaf(fabsf(v), -0.5f * kTanhA2, 0.5f) : table[at[k]];   // slope(-|z|)
            f[2 * w + k] = dy.get(2 * w + k) * (v < 0.f ? h : 1.f - h);
        }
    }
    if (most[0] > 0x7f80 || most[1] > 0x7f80) {   // a NaN stays one
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float v = z.get(i);
            f[i] = v != v ? v : f[i];
        }
    }
}

// Pass 1.  Workgroup: 128 columns of one strip of rows, of dz or (the last
// blocks) of x.  16 lanes hold a row's 128 columns, 16 rows at a time.  4096 x
// 28672 with 8192 columns of x: 98 us with gelu (5.4 TB/s), 500 x 2048 with 2048
// 4.7 us.  512 columns a row
// (whole waves, so that a row's maximum takes more lane exchanges) and strips of
// 64 to 1024 rows measured no faster.
template <int ACT, bool TABLE, bool NT>
__global__ void __launch_bounds__(kThreadsG)
grad_stats_kernel(Grad p) {
    __shared__ float s_table[TABLE ? kTableSize : 1];
    __shared__ float s_max[kRowLanes][kTileCols], s_sum[kRowLanes][kTileCols];
    const int cl = threadIdx.x % kColLanes, rl = threadIdx.x / kColLanes;
    const int per_part = p.blocks_n + p.blocks_k;
    const int part = blockIdx.x / per_part;
    const int block = blockIdx.x - part * per_part;
    const bool is_x = block >= p.blocks_n;
    const int cb = is_x ? block - p.blocks_n : block;
    const int64_t width = is_x ? p.K : p.N;
    const int64_t col = (int64_t)cb * kTileCols + cl * 8;
    const bool ok = col < width;                       // widths are multiples of 16
    const int64_t r1 = min(p.M, (part + 1) * p.strip);
    for (int64_t i = (int64_t)blockIdx.x * kThreadsG + threadIdx.x; i < p.num_counters;
         i += (int64_t)gridDim.x * kThreadsG)
        p.counters[i] = 0u;
    if (TABLE && !is_x) {
        fill_table<ACT>(s_table);
        __syncthreads();
    }
    float cmax[8], csum[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) cmax[i] = csum[i] = 0.f;
    for (int64_t r = part * p.strip + rl; r < r1; r += kRowLanes * kStatUnroll) {
        Raw8<bf16_t> a[kStatUnroll], b[kStatUnroll];
#pragma unroll
        for (int u = 0; u < kStatUnroll; ++u) {
            const int64_t row = r + u * kRowLanes;
            a[u].zero();
            b[u].zero();
            if (ok && row < r1) {
                a[u].template load<NT>((is_x ? p.x : p.dy) + row * width + col);
                if (ACT != kActNone && !is_x) b[u].template load<NT>(p.z + row * width + col);
            }
        }
#pragma unroll
        for (int u = 0; u < kStatUnroll; ++u) {
            float f[8];
            if (is_x) {
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = a[u].get(i);
            } else if constexpr (TABLE) {
                dz8_table(a[u], b[u], s_table, f);
            } else {
                dz8<ACT>(a[u], b[u], f);
            }
            float rmax = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                cmax[i] = fmaxf(cmax[i], fabsf(f[i]));
                rmax = fmaxf(rmax, fabsf(f[i]));
                csum[i] += f[i];
            }
            if (!is_x && p.want_rows) {
                const int64_t row = r + u * kRowLanes;
                rmax = row16_max(rmax);
                if (cl == 0 && row < r1) p.row_max[cb * p.M + row] = rmax;
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        s_max[rl][cl * 8 + i] = cmax[i];
        s_sum[rl][cl * 8 + i] = csum[i];
    }
    __syncthreads();
    const int t = threadIdx.x % kTileCols;
    const int64_t c = (int64_t)cb * kTileCols + t;
    if (c >= width) return;
    if (threadIdx.x < kTileCols) {
        float m = 0.f;
#pragma unroll
        for (int i = 0; i < kRowLanes; ++i) m = fmaxf(m, s_max[i][t]);
        (is_x ? p.x_max : p.col_max)[part * width + c] = m;
    } else if (!is_x) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kRowLanes; ++i) sum += s_sum[i][t];
        p.col_sum[part * width + c] = sum;
    }
}

// Pass 2.  Workgroup: 64 rows of dz, columns of dz or columns of x, 16 slices
// of their partial results each (4096 x 28672 with 8192: 6 us, 8 MB).
constexpr int kScaleThreads = 1024;

// (scale, its reciprocal)
__device__ __forceinline__ float2 scale_of(float amax, float qmax) {
    float s = amax / qmax;
    if (s < 0x1p-126f) s = 0.f;       // (its reciprocal would leave fp32)
    return float2{s, s == 0.f ? 0.f : 1.f / s};
}

__global__ void __launch_bounds__(kScaleThreads)
grad_scales_kernel(Grad p, int blocks_rows, int blocks_cols) {
    __shared__ float s_max[16][64], s_sum[16][64];
    const int lane = threadIdx.x % 64, slice = threadIdx.x / 64;
    int b = blockIdx.x;
    const float* part_max;
    const float* part_sum = nullptr;
    float* scale;
    int64_t n;
    int parts;
    float qmax = Fp8Fmt<1>::kMax;
    if (b < blocks_rows) {
        part_max = p.row_max; n = p.M; parts = p.blocks_n; scale = p.row_scale;
    } else if (b < blocks_rows + blocks_cols) {
        b -= blocks_rows;
        part_max = p.col_max; part_sum = p.dbias ? p.col_sum : nullptr; n = p.N; parts = p.parts;
        scale = p.col_scale;
    } else {
        b -= blocks_rows + blocks_cols;
        part_max = p.x_max; n = p.K; parts = p.parts; scale = p.x_scale; qmax = Fp8Fmt<0>::kMax;
    }
    const int64_t i = (int64_t)b * 64 + lane;
    float m = 0.f, sum = 0.f;
    if (i < n)
        for (int q0 = slice; q0 < parts; q0 += 16 * 8) {
            float v[8], w[8];   // loaded together: the pass is one memory latency or two long
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int q = q0 + 16 * k;
                v[k] = q < parts ? part_max[q * n + i] : 0.f;
                w[k] = part_sum && q < parts ? part_sum[q * n + i] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                m = fmaxf(m, v[k]);
                sum += w[k];
            }
        }
    s_max[slice][lane] = m;
    s_sum[slice][lane] = sum;
    __syncthreads();
    if (slice != 0 || i >= n) return;
#pragma unroll
    for (int q = 1; q < 16; ++q) {
        m = fmaxf(m, s_max[q][lane]);
        sum += s_sum[q][lane];
    }
    const float2 sr = scale_of(m, qmax);
    scale[i] = sr.x;
    scale[n + i] = sr.y;
    if (part_sum) p.dbias[i] = sum;
}

// A scale and its reciprocal (0 and 0 included) as the exact division takes them.
// It is proved for scales from 2^-60 on: a smaller one is lifted by 2^66, and so are
// the values that it divides (all of it exact: the quotients stay the same).
// Returns the values' factor.
__device__ __forceinline__ float lift(float2& sr) {
    if (!(sr.x > 0.f && sr.x < 0x1p-60f)) return 1.f;
    sr = float2{sr.x * 0x1p66f, sr.y * 0x1p-66f};
    return 0x1p66f;
}

// value / s: EXACT correctly rounded (s lifted, or from 2^-60 on), else the product
// by r = 1 / s.  With s = r = 0 every finite value gives 0, with s infinite (r = 0)
// an infinity gives NaN; NaN stays NaN.
template <bool EXACT>
__device__ __forceinline__ float over_scale(float v, float s, float r) {
    if constexpr (EXACT) return div_fast(v, Div{s, r, true});
    else return v * r;
}

// Pass 3.  Workgroup: a tile of ROWS rows x 128 columns of dz or (the last
// blocks) of x.  A thread takes 4 consecutive rows of 8 columns at a time, so
// that 4 codes of a column make one word of the transposed tile in LDS: 128
// rows of ROWS / 16 chunks of 16 bytes, chunk c of column n at
// c ^ ((n >> 3) % (ROWS / 16)), which spreads the 16 column lanes over the banks.
//
// Bound by memory at training sizes (4096 x 28672 with 8192 columns of x, gelu:
// 142 us, 5.7 TB/s), by latency at small ones (500 x 2048 with 2048: 8 us).
//
// JOIN: the workgroup joins the partial maxima of its columns and rows itself
// (at most kJoinParts of each), in place of pass 2; those of the first strip
// write the columns' scales and dbias, those of the first column block the
// rows' scales.
constexpr int kJoinParts = 64;

// f over the values p[0], p[n], ... of `parts` partial results, 32 loaded at a
// time (one memory latency; read one by one they cost 1347 x 3600 6 us).
template <class F>
__device__ __forceinline__ float join(const float* p, int64_t n, int parts, F f) {
    float acc = 0.f;
    for (int q0 = 0; q0 < parts; q0 += 32) {
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = q0 + k < parts ? p[(q0 + k) * n] : 0.f;
#pragma unroll
        for (int k = 0; k < 32; ++k) acc = f(acc, v[k]);
    }
    return acc;
}
__device__ __forceinline__ float larger(float a, float b) { return fmaxf(a, b); }
__device__ __forceinline__ float added(float a, float b) { return a + b; }

// ROWS: 128, or 64 (half the work a workgroup) where the grid is small.
template <int ACT, bool TABLE, bool JOIN, int ROWS, bool NT>
__global__ void __launch_bounds__(kThreadsG)
grad_quantize_kernel(Grad p) {
    constexpr int kChunks = ROWS / 16;           // of a transposed row
    __shared__ __attribute__((aligned(16))) uint32_t s_t[kTileCols][ROWS / 4];
    __shared__ __attribute__((aligned(16))) float s_col[3][kTileCols];   // scales, reciprocals, factors (lift())
    __shared__ float s_row[3][ROWS];
    __shared__ int s_lifted[kThreadsG / kWaveSize];
    __shared__ float s_table[TABLE ? kTableSize : 1];
    constexpr bool kExactDz = ACT == kActNone || ACT == kActRelu;
    const int cl = threadIdx.x % kColLanes, rl = threadIdx.x / kColLanes;
    const int per_strip = p.blocks_n + p.blocks_k;
    // Last strips first: they were pass 1's last, and what the caches still hold
    // of dy, z and x is theirs.
    const int64_t turn = blockIdx.x / per_strip;
    const int block = (int)(blockIdx.x - turn * per_strip);
    const int64_t strip = gridDim.x / per_strip - 1 - turn;
    const bool is_x = block >= p.blocks_n;
    const int cb = is_x ? block - p.blocks_n : block;
    const int64_t width = is_x ? p.K : p.N;
    const int64_t col = (int64_t)cb * kTileCols + cl * 8;
    const int64_t row0 = strip * ROWS;
    const bool ok = col < width;
    const bool transposed = is_x || p.want_cols;
    constexpr int kSteps = ROWS / (4 * kRowLanes);
    Raw8<bf16_t> a[kSteps][4], b[kSteps][4];
    auto fetch = [&](int it) __attribute__((always_inline)) {
        const int64_t r = row0 + (it * kRowLanes + rl) * 4;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            a[it][k].zero();
            b[it][k].zero();
            if (ok && r + k < p.M) {
                a[it][k].template load<NT>((is_x ? p.x : p.dy) + (r + k) * width + col);
                if (ACT != kActNone && !is_x) b[it][k].template load<NT>(p.z + (r + k) * width + col);
            }
        }
    };
    fetch(0);   // under way while the scales are found
    if (TABLE && !is_x) fill_table<ACT>(s_table);
    // Whether the exact division of this workgroup's values meets a lifted scale.
    int lifted = 0;
    {   // scales: the first 128 threads the columns', the others the rows'
        static_assert(kThreadsG >= kTileCols + ROWS, "one thread for each row and column");
        const int t = threadIdx.x % kTileCols;
        if (threadIdx.x < kTileCols) {
            const int64_t c = (int64_t)cb * kTileCols + t;
            float* scale = is_x ? p.x_scale : p.col_scale;
            float2 sr{0.f, 0.f};
            if (c < width) {
                if constexpr (JOIN) {
                    const float m = join((is_x ? p.x_max : p.col_max) + c, width, p.parts, larger);
                    sr = scale_of(m, is_x ? Fp8Fmt<0>::kMax : Fp8Fmt<1>::kMax);
                    if (strip == 0) {
                        scale[c] = sr.x;
                        if (!is_x && p.dbias) p.dbias[c] = join(p.col_sum + c, width, p.parts, added);
                    }
                } else {
                    sr = float2{scale[c], scale[width + c]};
                }
            }
            const float up = kExactDz || is_x ? lift(sr) : 1.f;
            lifted = up != 1.f;
            s_col[0][t] = sr.x;
            s_col[1][t] = sr.y;
            s_col[2][t] = up;
        } else if (t < ROWS) {
            const int64_t r = row0 + t;
            float2 sr{0.f, 0.f};
            if (!is_x && p.want_rows && r < p.M) {
                if constexpr (JOIN) {
                    sr = scale_of(join(p.row_max + r, p.M, p.blocks_n, larger), Fp8Fmt<1>::kMax);
                    if (block == 0) p.row_scale[r] = sr.x;
                } else {
                    sr = float2{p.row_scale[r], p.row_scale[p.M + r]};
                }
            }
            const float up = kExactDz ? lift(sr) : 1.f;
            lifted = up != 1.f;
            s_row[0][t] = sr.x;
            s_row[1][t] = sr.y;
            s_row[2][t] = up;
        }
        const bool any = __ballot(lifted) != 0;
        if (threadIdx.x % kWaveSize == 0) s_lifted[threadIdx.x / kWaveSize] = any;
        __syncthreads();
        static_assert(kThreadsG / kWaveSize == 4, "four waves' flags");
        lifted = __builtin_amdgcn_readfirstlane(s_lifted[0] | s_lifted[1] | s_lifted[2] | s_lifted[3]);
    }
    float cs[8], cr[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = s_col[0][cl * 8 + i];
        cr[i] = s_col[1][cl * 8 + i];
    }
#pragma unroll
    for (int it = 0; it < kSteps; ++it) {
        const int mg = it * kRowLanes + rl;            // group of 4 rows in the tile
        const int64_t r = row0 + mg * 4;
        if (it > 0) fetch(it);   // (a step ahead, the registers would cost a wave of four)
        float rs[4], rr[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            rs[k] = s_row[0][mg * 4 + k];
            rr[k] = s_row[1][mg * 4 + k];
        }
        float f[4][8];
        uint32_t words[8];
        const auto lift_columns = [&]() __attribute__((always_inline)) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[k][i] *= s_col[2][cl * 8 + i];
        };
        if (is_x) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[k][i] = a[it][k].get(i);
            if (lifted) lift_columns();
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int i = 0; i < 8; ++i) f[k][i] = over_scale<true>(f[k][i], cs[i], cr[i]);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int w = Fp8Fmt<0>::cvt_pk<false>(f[0][i], f[1][i], 0);
                words[i] = (uint32_t)Fp8Fmt<0>::cvt_pk<true>(f[2][i], f[3][i], w);
            }
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (TABLE) dz8_table(a[it][k], b[it][k], s_table, f[k]);
                else dz8<ACT>(a[it][k], b[it][k], f[k]);
            }
            if (p.want_rows) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float t[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = f[k][i];
                    if constexpr (kExactDz)
                        if (lifted)
#pragma unroll
                            for (int i = 0; i < 8; ++i) t[i] *= s_row[2][mg * 4 + k];
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] = over_scale<kExactDz>(t[i], rs[k], rr[k]);
                    u32x2 codes;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        int w = Fp8Fmt<1>::cvt_pk<false>(t[4 * h], t[4 * h + 1], 0);
                        codes[h] = (uint32_t)Fp8Fmt<1>::cvt_pk<true>(t[4 * h + 2], t[4 * h + 3], w);
                    }
                    if (ok && r + k < p.M)
                        store_hinted<NT>(reinterpret_cast<u32x2*>(p.q_rows + (r + k) * p.N + col), codes);
                }
            }
            if constexpr (kExactDz)
                if (lifted) lift_columns();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                int w = Fp8Fmt<1>::cvt_pk<false>(over_scale<kExactDz>(f[0][i], cs[i], cr[i]),
                                                 over_scale<kExactDz>(f[1][i], cs[i], cr[i]), 0);
                words[i] = (uint32_t)Fp8Fmt<1>::cvt_pk<true>(over_scale<kExactDz>(f[2][i], cs[i], cr[i]),
                                                             over_scale<kExactDz>(f[3][i], cs[i], cr[i]), w);
            }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s_t[cl * 8 + i][(((mg >> 2) ^ (cl % kChunks)) << 2) | (mg & 3)] = words[i];
    }
    if (!transposed) return;
    __syncthreads();
    uint8_t* out = is_x ? p.q_x : p.q_cols;
#pragma unroll
    for (int it = 0; it < kTileCols * kChunks / kThreadsG; ++it) {
        const int q = it * kThreadsG + threadIdx.x;
        const int n = q / kChunks, c = q % kChunks;
        const int64_t row = (int64_t)cb * kTileCols + n, m = row0 + c * 16;
        if (row < width && m < p.Mp)
            *reinterpret_cast<u32x4*>(out + row * p.Mp + m) =
                *reinterpret_cast<const u32x4*>(&s_t[n][(c ^ ((n >> 3) % kChunks)) << 2]);
    }
}

// n values of 0 (the gradients of a batch without rows).
__global__ void __launch_bounds__(kThreadsG) zero_fill_kernel(uint16_t* p, int64_t n) {
    for (int64_t i = blockIdx.x * (int64_t)kThreadsG + threadIdx.x; i < n; i += (int64_t)gridDim.x * kThreadsG)
        p[i] = 0;
}

// ---------------------------------------------------------------- host ---

int64_t up(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t align256(int64_t n) { return up(n, 256) * 256; }
bool at(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

constexpr int64_t kMaxDim = int64_t(1) << 23;
constexpr int64_t kCounterArea = int64_t(256) << 10;   // the multiply's arrival counters

int grad_shape(int64_t M, int64_t N, int64_t K, bool want_dw) {
    if (M < 0 || M > (want_dw ? kMaxDim : INT32_MAX) || N < 16 || N > kMaxDim || N % 16 != 0 || K < 16 ||
        K > kMaxDim || K % 16 != 0)
        return FP8MM_ERR_SHAPE;
    // One-dimensional grids of 128 x 128 tiles.
    if (up(M, kTileRows) * (up(N, kTileCols) + up(K, kTileCols)) > INT32_MAX) return FP8MM_ERR_SHAPE;
    return FP8MM_OK;
}

// Pass 3 joins the partial results itself where there are at most kJoinParts
// for a row (column blocks) and for a column (strips).
bool joins(const Grad& p) { return p.blocks_n <= kJoinParts && p.parts <= kJoinParts; }

// Rows of a strip of pass 1: 64 (one round of loads per thread), more where
// there are strips enough without that, up to 256, or where that leaves few
// enough strips for pass 3 to join.
int64_t strip_rows(int64_t M, int64_t blocks_n, int64_t blocks) {
    const int64_t round = kRowLanes * kStatUnroll;
    int64_t s = round;
    while (s < 256 && up(M, 2 * s) * blocks >= 2048) s *= 2;
    if (blocks_n <= kJoinParts && up(M, s) > kJoinParts) s = up(up(M, kJoinParts), round) * round;
    return s;
}

// The two products of a call (sizes only).
void products(int64_t M, int64_t N, int64_t K, int64_t Mp, fp8mm::Product (&q)[2]) {
    q[0] = fp8mm::Product{nullptr, nullptr, nullptr, nullptr, nullptr, M, K, N};
    q[1] = fp8mm::Product{nullptr, nullptr, nullptr, nullptr, nullptr, N, K, Mp};
}

struct GradSpace {
    int64_t mm, q_rows, q_cols, q_x, scales, partials, total;   // byte offsets
    Grad p;
};

// Everything about a call but its pointers.
GradSpace grad_space(int64_t M, int64_t N, int64_t K, bool want_dx, bool want_dw) {
    GradSpace g;
    Grad& p = g.p;
    p.M = M; p.N = N; p.K = K;
    p.Mp = M > 256 ? up(M, 64) * 64 : up(M, 16) * 16;
    p.want_rows = want_dx;
    p.want_cols = want_dw;
    p.blocks_n = (int)up(N, kTileCols);
    p.blocks_k = want_dw ? (int)up(K, kTileCols) : 0;
    p.strip = strip_rows(M, p.blocks_n, p.blocks_n + p.blocks_k);
    p.parts = (int)up(M, p.strip);
    int64_t mm = kCounterArea;
    if (want_dx && M > 0) {
        const int64_t n = fp8_scaled_mm_workspace_size(M, K, N, FP8MM_ROWWISE, 0, -1, 0);
        mm = n > mm ? n : mm;
    }
    if (want_dw && M > 0) {
        const int64_t n = fp8_scaled_mm_workspace_size(N, K, p.Mp, FP8MM_ROWWISE, 0, -1, 0);
        mm = n > mm ? n : mm;
    }
    if (want_dx && want_dw && M > 0) {
        fp8mm::Product q[2];
        products(M, N, K, p.Mp, q);
        const fp8mm::PairPlan plan = fp8mm::plan_pair(q);
        const int64_t n = plan.cfg >= 0 ? fp8mm::pair_workspace(q, plan) : 0;
        mm = n > mm ? n : mm;
    }
    g.mm = align256(mm);
    g.q_rows = g.mm;
    g.q_cols = g.q_rows + (want_dx ? align256(M * N) : 0);
    g.q_x = g.q_cols + (want_dw ? align256(N * p.Mp) : 0);
    g.scales = g.q_x + (want_dw ? align256(K * p.Mp) : 0);
    g.partials = g.scales + align256(8 * (M + N + K));
    g.total = g.partials + align256(4 * ((want_dx ? p.blocks_n * M : 0) + 2 * p.parts * N + p.parts * K));
    return g;
}

// Tiles of 128 rows below which 64 rows a workgroup are faster.
constexpr int64_t kSmallGrid = 512;

// NT: for inputs beyond the memory-side cache, which pass 3 would not find there
// (the whole gradient of 4096 x 28672 x 8192 on one MI355X, us without and with:
// gelu 1631 and 1612, relu 1572 and 1545; where they fit, 1000 x 4000 x 2000,
// 50.0 and 51.5).
template <int ACT, bool TABLE, bool NT>
void launch_passes(const Grad& p, hipStream_t hs) {
    const int per = p.blocks_n + p.blocks_k;
    const int64_t tiles = up(p.M, kTileRows) * per;
    const dim3 block(kThreadsG);
    hipLaunchKernelGGL((grad_stats_kernel<ACT, TABLE, NT>), dim3((unsigned)(p.parts * per)), block, 0, hs, p);
    const bool join = joins(p);
    if (!join || !(p.want_rows || p.want_cols)) {
        const int rows = p.want_rows ? (int)up(p.M, 64) : 0, cols = (int)up(p.N, 64);
        const int xs = p.blocks_k ? (int)up(p.K, 64) : 0;
        hipLaunchKernelGGL(grad_scales_kernel, dim3((unsigned)(rows + cols + xs)), dim3(kScaleThreads), 0, hs, p,
                           rows, cols);
    }
    if (!(p.want_rows || p.want_cols)) return;
    if (!join)
        hipLaunchKernelGGL((grad_quantize_kernel<ACT, TABLE, false, kTileRows, NT>), dim3((unsigned)tiles), block, 0, hs, p);
    else if (tiles >= kSmallGrid)
        hipLaunchKernelGGL((grad_quantize_kernel<ACT, TABLE, true, kTileRows, NT>), dim3((unsigned)tiles), block, 0, hs, p);
    else
        hipLaunchKernelGGL((grad_quantize_kernel<ACT, false, true, 64, false>), dim3((unsigned)(up(p.M, 64) * per)), block, 0, hs, p);
}

template <int ACT>
void launch_passes(const Grad& p, hipStream_t hs) {
    const int64_t bytes = 2 * p.M * ((ACT == kActNone ? 1 : 2) * p.N + (p.blocks_k ? p.K : 0));
    const bool stream = bytes > kCachedBytes;
    if constexpr (kHasTable<ACT>) {
        // (dz has tiles enough to be bound by its arithmetic.)
        if (up(p.M, kTileRows) * p.blocks_n >= kSmallGrid)
            return stream ? launch_passes<ACT, true, true>(p, hs) : launch_passes<ACT, true, false>(p, hs);
    }
    if (stream) launch_passes<ACT, false, true>(p, hs);
    else launch_passes<ACT, false, false>(p, hs);
}

}  // namespace

extern "C" {

int64_t fp8_linear_backward_workspace_size(int64_t M, int64_t N, int64_t K, int want_dx, int want_dw) {
    if (grad_shape(M, N, K, want_dw != 0) != FP8MM_OK) return -1;
    return grad_space(M, N, K, want_dx != 0, want_dw != 0).total;
}

int fp8_linear_backward(const void* dy, const void* x, const void* wt, int wt_format, const float* wt_scale,
                        const void* z, int activation, void* dx, void* dw, float* dbias, int64_t M, int64_t N,
                        int64_t K, struct ihipStream_t* stream, void* workspace, int64_t workspace_bytes) {
    if (activation < FP8MM_ACT_NONE || activation > FP8MM_ACT_SILU) return FP8MM_ERR_ACTIVATION;
    if (dx && wt_format != FP8MM_E4M3FN && wt_format != FP8MM_E5M2) return FP8MM_ERR_FORMAT;
    int st = grad_shape(M, N, K, dw != nullptr);
    if (st != FP8MM_OK) return st;
    if (!dx && !dw && !dbias && M > 0) return FP8MM_ERR_NULL;
    if (M > 0 && (!dy || (activation != FP8MM_ACT_NONE && !z) || (dx && (!wt || !wt_scale)) || (dw && !x)))
        return FP8MM_ERR_NULL;
    if (!at(dy, 2) || !at(z, 2) || !at(x, 2) || !at(dx, 2) || !at(dw, 2) || !at(dbias, 4) || !at(wt, 16) ||
        !at(wt_scale, 4) || !at(workspace, 256))
        return FP8MM_ERR_ALIGN;
    GradSpace g = grad_space(M, N, K, dx != nullptr, dw != nullptr);
    if (M > 0 && (!workspace || workspace_bytes < g.total)) return FP8MM_ERR_WORKSPACE;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return FP8MM_ERR_DEVICE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    (void)hipGetLastError();
    if (M == 0) {
        if (dw)
            hipLaunchKernelGGL(zero_fill_kernel, dim3(2048), dim3(kThreadsG), 0, hs, static_cast<uint16_t*>(dw), N * K);
        if (dbias)
            hipLaunchKernelGGL(zero_fill_kernel, dim3(64), dim3(kThreadsG), 0, hs, reinterpret_cast<uint16_t*>(dbias),
                               2 * N);
        return hipGetLastError() == hipSuccess ? FP8MM_OK : FP8MM_ERR_LAUNCH;
    }
    std::lock_guard<std::mutex> together(fp8mm::enqueue_lock(workspace));
    char* ws = static_cast<char*>(workspace);
    Grad& p = g.p;
    p.dy = static_cast<const bf16_t*>(dy);
    p.z = static_cast<const bf16_t*>(z);
    p.x = static_cast<const bf16_t*>(x);
    p.q_rows = reinterpret_cast<uint8_t*>(ws + g.q_rows);
    p.q_cols = reinterpret_cast<uint8_t*>(ws + g.q_cols);
    p.q_x = reinterpret_cast<uint8_t*>(ws + g.q_x);
    p.row_scale = reinterpret_cast<float*>(ws + g.scales);
    p.col_scale = p.row_scale + 2 * M;
    p.x_scale = p.col_scale + 2 * N;
    p.col_max = reinterpret_cast<float*>(ws + g.partials);
    p.col_sum = p.col_max + p.parts * N;
    p.x_max = p.col_sum + p.parts * N;
    p.row_max = p.x_max + p.parts * K;
    p.dbias = dbias;
    fp8mm::Product q[2];
    products(M, N, K, p.Mp, q);
    fp8mm::PairPlan pair{-1, {1, 1}};
    if (dx && dw && wt_format == FP8MM_E4M3FN) pair = fp8mm::plan_pair(q);
    p.counters = reinterpret_cast<uint32_t*>(ws);
    if (pair.cfg >= 0) {
        p.num_counters = fp8mm::pair_counters(q, pair);
    } else {
        const int of_dx = dx ? fp8mm::product_counters(q[0]) : 0, of_dw = dw ? fp8mm::product_counters(q[1]) : 0;
        p.num_counters = of_dx > of_dw ? of_dx : of_dw;   // (a product leaves its counters at zero)
    }
    switch (activation) {
        case kActRelu: launch_passes<kActRelu>(p, hs); break;
        case kActGelu: launch_passes<kActGelu>(p, hs); break;
        case kActGeluTanh: launch_passes<kActGeluTanh>(p, hs); break;
        case kActSilu: launch_passes<kActSilu>(p, hs); break;
        default: launch_passes<kActNone>(p, hs); break;
    }
    if (hipGetLastError() != hipSuccess) return FP8MM_ERR_LAUNCH;
    if (pair.cfg >= 0) {
        q[0] = fp8mm::Product{p.q_rows, wt, p.row_scale, wt_scale, dx, M, K, N};
        q[1] = fp8mm::Product{p.q_cols, p.q_x, p.col_scale, p.x_scale, dw, N, K, p.Mp};
        return fp8mm::run_pair(q, pair, hs, ws);
    }
    if (dx) {
        st = fp8_scaled_mm_typed(p.q_rows, FP8MM_E5M2, wt, wt_format, p.row_scale, wt_scale, nullptr, dx, M, K, N,
                                 FP8MM_ROWWISE, stream, -1, 0, ws, g.mm);
        if (st != FP8MM_OK) return st;
    }
    if (dw)
        st = fp8_scaled_mm_typed(p.q_cols, FP8MM_E5M2, p.q_x, FP8MM_E4M3FN, p.col_scale, p.x_scale, nullptr, dw, N,
                                 K, p.Mp, FP8MM_ROWWISE, stream, -1, 0, ws, g.mm);
    return st;
}

}  // extern "C"
