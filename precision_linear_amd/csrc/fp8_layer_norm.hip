// Layer norm and its gradient for gfx950 (MI355X), with the float8
// quantisation of the normalised rows (formulas: include/fp8_layer_norm.h).
//
// HBM-bound: every element is read once and written once.  A row stays in
// registers between its statistics and its output.
//
// Layout: a row belongs to W waves (W = ceil(cols / 1024), at most 16); lane t
// of them holds V = 2 vectors of 8 consecutive elements, vectors t and
// t + 64 W, and where cols is no multiple of 8 the first cols % 8 lanes hold
// one element more.  A thread's columns are the same for every row it meets, so
// w and b (8 bytes of parameters to 2 bytes of bf16 x) and, in the gradient,
// the sums of dw and db stay in registers over the workgroup's rows.  Rows of
// more than 16384 + 7 elements take the *_long kernels, which sweep the row
// (from L2) instead of holding it.
//
// Rows that do not start on a 16-byte boundary (cols % 8 != 0) are read and
// written with the same 16-byte instructions: global memory takes any 2-byte
// aligned address.
//
// Non-temporal hints: bf16 calls that move more than the memory-side cache holds
// take them on the loads, on the codes and, in long rows, on dx; each load and
// store was measured on its own.  us on one MI355X, without and with: forward
// with y and codes 16384 x 8192 134 and 126, 32768 x 4096 142 and 112, 65536 x
// 1024 64 and 59; y alone 16384 x 8192 97 and 83; gradient with a residual 16384
// x 8192 201 and 183, 65536 x 1024 108 and 93.  With the hint on y as well the
// forward's gain is lost (32768 x 4096 137, y alone 89).  Smaller calls find
// their inputs in the cache and lose with it (4095 x 4097 14.5 and 20.0).  fp32
// loses too (gradient 8192 x 8192 198 and 212): a lane's two 16-byte halves lie
// in lines that it shares with its neighbours.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <cmath>
#include <type_traits>

#include "../../include/fp8_layer_norm.h"
#include "enqueue_lock.h"
#include "fp8_convert.h"
#include "lane_ops.h"

namespace {

constexpr int kVecs = 2;                     // vectors of 8 elements per lane
constexpr int kMaxWaves = 16;                // waves per row (and per workgroup)
constexpr int64_t kHeldCols = (int64_t)kMaxWaves * kWaveSize * kVecs * 8 + 7;
constexpr int kLongThreads = 1024;

// w or b at column c .. c + 7 (fp32 or bf16; null: `none`).
__device__ __forceinline__ void load_param8(const void* p, int bf16, int64_t c, float none, float (&f)[8]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = none;
    } else if (bf16) {
        Raw8<bf16_t> r;
        r.load(static_cast<const bf16_t*>(p) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = r.get(i);
    } else {
        Raw8<float> r;
        r.load(static_cast<const float*>(p) + c);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = r.get(i);
    }
}
__device__ __forceinline__ float load_param1(const void* p, int bf16, int64_t c, float none) {
    if (!p) return none;
    return bf16 ? load1(static_cast<const bf16_t*>(p) + c) : load1(static_cast<const float*>(p) + c);
}

// ------------------------------------------------------------- forward ---

struct LnFwd {
    const void* x;
    const void* w;
    const void* b;
    int param_bf16;
    float eps;
    void* y;
    uint8_t* q;
    int q_format;
    float* scale;
    float* mean;
    float* rstd;
    int64_t rows;
    int64_t cols;
    int waves;   // W, waves per row
};

// 8 codes of y / scale.  `slow` covers scales outside the fast division's
// range: 0 (every finite y is 0 or rounds to it), tiny, infinite and NaN ones.
template <int FMT>
__device__ __forceinline__ u32x2 codes8(const float (&y)[8], const Div& d) {
    float t[8];
    if (d.fast) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = div_fast(y[i], d);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[i] = d.s == 0.f ? fabsf(y[i]) : quant1<FMT, false>(y[i], d);
    }
    u32x2 out;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int pk = Fp8Fmt<FMT>::template cvt_pk<false>(t[4 * h], t[4 * h + 1], 0);
        pk = Fp8Fmt<FMT>::template cvt_pk<true>(t[4 * h + 2], t[4 * h + 3], pk);
        out[h] = (uint32_t)pk;
    }
    return out;
}

// 1 / sqrt(variance + eps).  Squares beyond the fp32 range give NaN, not the 0 that
// would make every y of the row b.
__device__ __forceinline__ float inverse_spread(float variance, float eps) {
    return variance < __builtin_inff() ? 1.f / sqrtf(variance + eps) : __builtin_nanf("");
}

// The scale of a row from its largest |y| (NaN skipped): a row whose statistics
// are NaN, or whose rstd is infinite (no variance, no eps: every y is 0 times
// that), gets a NaN scale, not the 0 of an empty maximum.
template <int FMT>
__device__ __forceinline__ float row_scale(float amax, float rstd) {
    return rstd < __builtin_inff() ? amax / Fp8Fmt<FMT>::kMax : __builtin_nanf("");
}

// One row per W waves.  WIDE: the workgroup is the row's W > 1 waves, which
// meet in LDS; otherwise each wave has a row of its own.  The next row is loaded
// while this one is worked on.  Bound by memory from about 10^7 elements on:
// y and codes 16384 x 8192 bf16 126 us (5.3 TB/s), 65536 x 1024 59 us (5.7); y
// alone 8192 x 8192 fp32 98 us (5.5); a large copy reaches 5.4.  One row: 3.7 us,
// two meetings of the waves between a load and a store.
//
// Variance: each wave takes the mean of its own share and the squares around
// that mean, and the shares are joined with
//   M2 = sum_w( M2_w + n_w (mean_w - mean)^2 )
// (T. Chan, G. Golub, R. LeVeque, 1979), which costs one meeting of the waves
// and loses nothing to a mean far from 0.
template <class T, bool WIDE, bool NT>
__global__ void __launch_bounds__(kMaxWaves* kWaveSize)
ln_forward_kernel(LnFwd p) {
    __shared__ float2 s_mom[2][kMaxWaves];
    __shared__ float s_max[2][kMaxWaves];
    const int lane = threadIdx.x % kWaveSize;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const int W = WIDE ? p.waves : 1;
    const int t = WIDE ? (int)threadIdx.x : lane;          // lane of the row
    const int tw = W * kWaveSize;
    const int cols = (int)p.cols;
    const int nv = cols / 8;                               // whole vectors in a row
    const bool has_tail = t < cols % 8;
    const int ct = nv * 8 + t;                             // this lane's tail column
    bool ok[kVecs];
    float w[kVecs][8], b[kVecs][8], wt = 0.f, bt = 0.f;
    int cnt = 0;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        ok[v] = t + v * tw < nv;
        cnt += 8 * __popcll(__ballot(ok[v]));
    }
    cnt += __popcll(__ballot(has_tail));
    const float n_w = (float)cnt;
    const float inv_nw = cnt ? 1.f / n_w : 0.f;
    const float inv_n = 1.f / (float)cols;

    const T* x = static_cast<const T*>(p.x);
    T* y = static_cast<T*>(p.y);
    const int64_t first = WIDE ? blockIdx.x : (int64_t)blockIdx.x * (blockDim.x / kWaveSize) + wave;
    const int64_t step = WIDE ? gridDim.x : (int64_t)gridDim.x * (blockDim.x / kWaveSize);

    Raw8<T> next[kVecs];
    float next_t = 0.f;
    auto fetch = [&](int64_t r) {
        const T* xr = x + r * p.cols;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            if (ok[v]) next[v].template load<NT>(xr + (t + v * tw) * 8);
        if (has_tail) next_t = load1(xr + ct);
    };
#pragma unroll
    for (int v = 0; v < kVecs; ++v) next[v].zero();
    if (first < p.rows) fetch(first);
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        if (ok[v]) {
            load_param8(p.w, p.param_bf16, (t + v * tw) * 8, 1.f, w[v]);
            load_param8(p.b, p.param_bf16, (t + v * tw) * 8, 0.f, b[v]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) w[v][i] = b[v][i] = 0.f;
        }
    }
    if (has_tail) {
        wt = load_param1(p.w, p.param_bf16, ct, 1.f);
        bt = load_param1(p.b, p.param_bf16, ct, 0.f);
    }

    int parity = 0;
    for (int64_t r = first; r < p.rows; r += step, parity ^= 1) {
        float f[kVecs][8], ft = next_t;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) f[v][i] = next[v].get(i);
        if (r + step < p.rows) fetch(r + step);

        float s = ft;   // lanes and vectors without elements hold zeros
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) s += f[v][i];
        s = wave_sum(s);
        const float m_w = s * inv_nw;
        float m2 = 0.f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
            if (ok[v])
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = f[v][i] - m_w;
                    m2 = fmaf(d, d, m2);
                }
        if (has_tail) m2 = fmaf(ft - m_w, ft - m_w, m2);
        m2 = wave_sum(m2);
        float mean = m_w;
        if constexpr (WIDE) {
            if (lane == 0) s_mom[parity][wave] = float2{s, m2};
            __syncthreads();
            // Lane l of each 16 takes wave l's share.
            const int l = lane % 16;
            const float2 mom = l < W ? s_mom[parity][l] : float2{0.f, 0.f};
            mean = lane_value(row16_sum(mom.x), 0) * inv_n;
            int c = 0;       // elements of wave l
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                c += 8 * min(kWaveSize, max(0, nv - v * tw - l * kWaveSize));
            c += l == 0 ? cols % 8 : 0;
            const float d = c ? mom.x / (float)c - mean : 0.f;
            m2 = lane_value(row16_sum(l < W ? fmaf((float)c * d, d, mom.y) : 0.f), 0);
        }
        const float rstd = inverse_spread(m2 * inv_n, p.eps);

        float amax = 0.f;
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[v][i] = fmaf((f[v][i] - mean) * rstd, w[v][i], b[v][i]);
                if (ok[v]) amax = fmaxf(amax, fabsf(f[v][i]));
            }
        ft = fmaf((ft - mean) * rstd, wt, bt);
        if (p.y) {
            T* yr = y + r * p.cols;
#pragma unroll
            for (int v = 0; v < kVecs; ++v)
                if (ok[v]) store8(yr + (t + v * tw) * 8, f[v]);
            if (has_tail) store1(yr + ct, ft);
        }
        if (p.q) {   // cols % 16 == 0: no tail
            amax = wave_max(amax);
            if constexpr (WIDE) {
                if (lane == 0) s_max[parity][wave] = amax;
                __syncthreads();
                amax = lane_value(row16_max(lane % 16 < W ? s_max[parity][lane % 16] : 0.f), 0);
            }
            uint8_t* qr = p.q + r * p.cols;
            auto write = [&](auto fmt) {
                constexpr int FMT = decltype(fmt)::value;
                const float sc = row_scale<FMT>(amax, rstd);
                if (t == 0) p.scale[r] = sc;
                const Div d = make_div(sc);
#pragma unroll
                for (int v = 0; v < kVecs; ++v)
                    if (ok[v])
                        store_hinted<NT>(reinterpret_cast<u32x2*>(qr + (t + v * tw) * 8), codes8<FMT>(f[v], d));
            };
            if (p.q_format == FP8LN_E4M3FN) write(std::integral_constant<int, 0>{});
            else write(std::integral_constant<int, 1>{});
        }
        if (p.mean && t == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

// Sum and maximum over a workgroup of kLongThreads (every thread returns them).
__device__ __forceinline__ float block_sum(float x, float* red) {
    x = wave_sum(x);
    __syncthreads();   // red may still be read by the last reduction
    if (threadIdx.x % kWaveSize == 0) red[threadIdx.x / kWaveSize] = x;
    __syncthreads();
    return lane_value(row16_sum(red[threadIdx.x % 16]), 0);
}
__device__ __forceinline__ float block_maximum(float x, float* red) {
    x = wave_max(x);
    __syncthreads();
    if (threadIdx.x % kWaveSize == 0) red[threadIdx.x / kWaveSize] = x;
    __syncthreads();
    return lane_value(row16_max(red[threadIdx.x % 16]), 0);
}

// Calls f(column, count) for this thread's vectors of 8 columns and, for the
// last cols % 8 columns, single ones.
template <class F8, class F1>
__device__ __forceinline__ void for_columns(int64_t cols, F8 f8, F1 f1) {
    const int64_t nv = cols / 8;
    for (int64_t g = threadIdx.x; g < nv; g += kLongThreads) f8(g * 8);
    if (threadIdx.x < cols % 8) f1(nv * 8 + threadIdx.x);
}

// Rows of any length, one workgroup each, swept once per step of the formula
// (sum, squares, y with its maximum, codes).  Bound by the L2: each sweep over y
// reads the parameters, four bytes for one of x (4096 x 32768 bf16, y and codes,
// 250 to 282 us by the card; on the latter 321 with y and its maximum in sweeps of
// their own).
template <class T>
__global__ void __launch_bounds__(kLongThreads)
ln_forward_long_kernel(LnFwd p) {
    __shared__ float red[kMaxWaves];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* xr = static_cast<const T*>(p.x) + r * p.cols;
        float s = 0.f;
        for_columns(p.cols,
                    [&](int64_t c) {
                        Raw8<T> v;
                        v.load(xr + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) s += v.get(i);
                    },
                    [&](int64_t c) { s += load1(xr + c); });
        const float mean = block_sum(s, red) / (float)p.cols;
        float m2 = 0.f;
        for_columns(p.cols,
                    [&](int64_t c) {
                        Raw8<T> v;
                        v.load(xr + c);
#pragma unroll
                        for (int i = 0; i < 8; ++i) m2 = fmaf(v.get(i) - mean, v.get(i) - mean, m2);
                    },
                    [&](int64_t c) { m2 = fmaf(load1(xr + c) - mean, load1(xr + c) - mean, m2); });
        const float rstd = inverse_spread(block_sum(m2, red) / (float)p.cols, p.eps);
        auto y8 = [&](int64_t c, float (&f)[8]) {
            Raw8<T> v;
            float w[8], b[8];
            v.load(xr + c);
            load_param8(p.w, p.param_bf16, c, 1.f, w);
            load_param8(p.b, p.param_bf16, c, 0.f, b);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = fmaf((v.get(i) - mean) * rstd, w[i], b[i]);
        };
        float amax = 0.f;
        T* yr = p.y ? static_cast<T*>(p.y) + r * p.cols : nullptr;
        for_columns(p.cols,
                    [&](int64_t c) {
                        float f[8];
                        y8(c, f);
                        if (yr) store8(yr + c, f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
                    },
                    [&](int64_t c) {   // (no codes then: cols % 16 != 0)
                        store1(yr + c, fmaf((load1(xr + c) - mean) * rstd, load_param1(p.w, p.param_bf16, c, 1.f),
                                            load_param1(p.b, p.param_bf16, c, 0.f)));
                    });
        if (p.q) {
            amax = block_maximum(amax, red);
            uint8_t* qr = p.q + r * p.cols;
            auto write = [&](auto fmt) {
                constexpr int FMT = decltype(fmt)::value;
                const float sc = row_scale<FMT>(amax, rstd);
                if (threadIdx.x == 0) p.scale[r] = sc;
                const Div d = make_div(sc);
                for_columns(p.cols,
                            [&](int64_t c) {
                                float f[8];
                                y8(c, f);
                                *reinterpret_cast<u32x2*>(qr + c) = codes8<FMT>(f, d);
                            },
                            [&](int64_t) {});
            };
            if (p.q_format == FP8LN_E4M3FN) write(std::integral_constant<int, 0>{});
            else write(std::integral_constant<int, 1>{});
        }
        if (p.mean && threadIdx.x == 0) {
            p.mean[r] = mean;
            p.rstd[r] = rstd;
        }
    }
}

// ------------------------------------------------------------ backward ---

struct LnBwd {
    const void* dy;
    const void* x;
    const float* mean;
    const float* rstd;
    const void* w;
    int param_bf16;
    const void* res;   // residual gradient, may be null
    void* dx;
    float* partial;    // [2][parts][pitch]: sums of dy * xh, then of dy
    int64_t rows;
    int64_t cols;
    int64_t pitch;
    int waves;         // W
    int subs;          // rows a workgroup works on at a time
};

// A lane's share of the columns: V vectors of 8 and at most one tail column.
template <int V>
struct Share {
    int t, tw;          // lane of the row, lanes of a row
    bool ok[V];
    bool has_tail;
    int tail;           // column
    __device__ __forceinline__ Share(int lane_of_row, int lanes, int cols)
        : t(lane_of_row), tw(lanes), has_tail(lane_of_row < cols % 8), tail(cols / 8 * 8 + lane_of_row) {
#pragma unroll
        for (int v = 0; v < V; ++v) ok[v] = t + v * tw < cols / 8;
    }
    __device__ __forceinline__ int col(int v) const { return (t + v * tw) * 8; }
};

// Which of a gradient's accesses take the non-temporal hint.
enum Stream { kStreamNone = 0, kStreamLoads = 1, kStreamAll = 2 };

// The rows blk * subs, + blocks * subs, ... of dx, `subs` rows at a time, W waves
// each.  SUMS: dw and db over these rows are added to the sums given.
template <class T, int V, bool SUMS, int NT>
__device__ __forceinline__ void backward_rows(const LnBwd& p, const Share<V>& c, int blk, int blocks,
                                              float (&dw)[V][8], float (&db)[V][8], float& dwt, float& dbt) {
    __shared__ float2 s_sum[2][kMaxWaves];
    const int lane = threadIdx.x % kWaveSize;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const int W = p.waves;
    const int sub = wave / W;
    const float inv_n = 1.f / (float)(int)p.cols;
    float w[V][8], wt = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[v][i] = 0.f;
        if (c.ok[v]) load_param8(p.w, p.param_bf16, c.col(v), 1.f, w[v]);
    }
    if (c.has_tail) wt = load_param1(p.w, p.param_bf16, c.tail, 1.f);
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    const T* res = static_cast<const T*>(p.res);
    T* dx = static_cast<T*>(p.dx);
    const int64_t step = (int64_t)blocks * p.subs;
    // The residual is loaded with the row where registers allow.
    constexpr bool kResEarly = V * sizeof(T) <= 4;
    int parity = 0;
    // Every sub goes through the same number of steps (they share barriers);
    // past the last row it works on zeros and stores nothing.
    for (int64_t base = (int64_t)blk * p.subs; base < p.rows; base += step, parity ^= 1) {
        const int64_t r = base + sub;
        const bool live = r < p.rows;
        Raw8<T> rx[V], rdy[V], rr[V];
        float xt = 0.f, dyt = 0.f, rt = 0.f;
        float mean = 0.f, rstd = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            rx[v].zero();
            rdy[v].zero();
            rr[v].zero();
        }
        const int64_t off = r * p.cols;
        if (live) {
            mean = p.mean[r];
            rstd = p.rstd[r];
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (c.ok[v]) {
                    rx[v].template load<NT != kStreamNone>(x + off + c.col(v));
                    rdy[v].template load<NT != kStreamNone>(dy + off + c.col(v));
                    if (kResEarly && res) rr[v].template load<NT != kStreamNone>(res + off + c.col(v));
                }
            if (c.has_tail) {
                xt = load1(x + off + c.tail);
                dyt = load1(dy + off + c.tail);
                if (res) rt = load1(res + off + c.tail);
            }
        }
        float s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c.ok[v])
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float d = rdy[v].get(i);
                    const float xh = (rx[v].get(i) - mean) * rstd;
                    const float g = d * w[v][i];
                    s1 += g;
                    s2 = fmaf(g, xh, s2);
                    if constexpr (SUMS) {
                        dw[v][i] = fmaf(d, xh, dw[v][i]);
                        db[v][i] += d;
                    }
                }
        const float xht = (xt - mean) * rstd;
        if (c.has_tail) {
            const float g = dyt * wt;
            s1 += g;
            s2 = fmaf(g, xht, s2);
            if constexpr (SUMS) {
                dwt = fmaf(dyt, xht, dwt);
                dbt += dyt;
            }
        }
        s1 = wave_sum(s1);
        s2 = wave_sum(s2);
        if (W > 1) {
            if (lane == 0) s_sum[parity][wave] = float2{s1, s2};
            __syncthreads();
            const int l = lane % 16;
            const float2 o = l < W ? s_sum[parity][sub * W + l] : float2{0.f, 0.f};
            s1 = lane_value(row16_sum(o.x), 0);
            s2 = lane_value(row16_sum(o.y), 0);
        }
        if (!live) continue;
        const float c1 = s1 * inv_n, c2 = s2 * inv_n;
        if (!kResEarly && res)
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (c.ok[v]) rr[v].template load<NT != kStreamNone>(res + off + c.col(v));
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c.ok[v]) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float xh = (rx[v].get(i) - mean) * rstd;
                    const float g = rdy[v].get(i) * w[v][i];
                    f[i] = fmaf(rstd, g - c1 - xh * c2, rr[v].get(i));
                }
                store8<NT == kStreamAll>(dx + off + c.col(v), f);
            }
        if (c.has_tail) store1(dx + off + c.tail, fmaf(rstd, dyt * wt - c1 - xht * c2, rt));
    }
}

// Bound by memory: with a residual 16384 x 8192 bf16 178 us (6.0 TB/s; three
// streams read to one written), 65536 x 1024 92 us (5.9), 8192 x 8192 fp32 194 us
// (5.5).
//
// dx, and this workgroup's share of dw and db: the sums over a workgroup's rows
// stay in registers and meet in LDS at the end (a fixed tree over the subs), so
// a workgroup writes one partial row.
template <class T, int V, int NT>
__global__ void __launch_bounds__(kMaxWaves* kWaveSize)
ln_backward_kernel(LnBwd p) {
    extern __shared__ float4 s_cols[];            // [subs / 2][dw, db][V][2][lanes of a row]
    __shared__ float s_tail[kMaxWaves / 2][2][8];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWaveSize);
    const int sub = wave / p.waves;
    const int tw = p.waves * kWaveSize;
    const Share<V> c((int)threadIdx.x - sub * tw, tw, (int)p.cols);
    float dw[V][8], db[V][8], dwt = 0.f, dbt = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dw[v][i] = db[v][i] = 0.f;
    backward_rows<T, V, true, NT>(p, c, blockIdx.x, gridDim.x, dw, db, dwt, dbt);

    // Join the subs: the upper half of them hands its sums to the lower half.
    // Lane t's four values of a vector's half h lie at [v][h][t]: no two lanes
    // meet in a bank.
    for (int n = p.subs; n > 1;) {
        const int half = (n + 1) / 2;
        const int slot = sub >= half ? sub - half : sub;
        float4* at = s_cols + (int64_t)slot * 4 * V * tw + c.t;
        __syncthreads();
        if (sub >= half && sub < n) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    at[(v * 2 + h) * tw] = float4{dw[v][4 * h], dw[v][4 * h + 1], dw[v][4 * h + 2], dw[v][4 * h + 3]};
                    at[((V + v) * 2 + h) * tw] =
                        float4{db[v][4 * h], db[v][4 * h + 1], db[v][4 * h + 2], db[v][4 * h + 3]};
                }
            if (c.has_tail) {
                s_tail[slot][0][c.t] = dwt;
                s_tail[slot][1][c.t] = dbt;
            }
        }
        __syncthreads();
        if (sub < n - half) {
#pragma unroll
            for (int v = 0; v < V; ++v)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const float4 a = at[(v * 2 + h) * tw], b = at[((V + v) * 2 + h) * tw];
                    dw[v][4 * h] += a.x;
                    dw[v][4 * h + 1] += a.y;
                    dw[v][4 * h + 2] += a.z;
                    dw[v][4 * h + 3] += a.w;
                    db[v][4 * h] += b.x;
                    db[v][4 * h + 1] += b.y;
                    db[v][4 * h + 2] += b.z;
                    db[v][4 * h + 3] += b.w;
                }
            if (c.has_tail) {
                dwt += s_tail[slot][0][c.t];
                dbt += s_tail[slot][1][c.t];
            }
        }
        n = half;
    }
    if (sub == 0) {
        float* pw = p.partial + blockIdx.x * p.pitch;
        float* pb = pw + gridDim.x * p.pitch;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (c.ok[v]) {
                store8(pw + c.col(v), dw[v]);
                store8(pb + c.col(v), db[v]);
            }
        if (c.has_tail) {
            pw[c.tail] = dwt;
            pb[c.tail] = dbt;
        }
    }
}

// Few rows: one launch, no partial results.  The first row_blocks workgroups
// write dx; the others take 64 columns each and sum dw and db over all the
// rows, reading dy and x again (from L2, where the first have just brought
// them): 16 lanes of 4 columns, blockDim / 16 slices of the rows, joined in a
// fixed order.  64 x 8192 with a residual 5.6 us in fp32, 4.4 in bf16: a launch
// and three memory latencies.
template <class T>
__device__ __forceinline__ void load4(const T* row, int64_t c, int64_t cols, float (&f)[4]) {
    if (c + 3 < cols) {
        if constexpr (sizeof(T) == 2) {
            typedef u32x2 u32x2_a2 __attribute__((aligned(2)));
            const u32x2 v = *reinterpret_cast<const u32x2_a2*>(row + c);
            f[0] = bf16_lo(v[0]);
            f[1] = bf16_hi(v[0]);
            f[2] = bf16_lo(v[1]);
            f[3] = bf16_hi(v[1]);
        } else {
            const u32x4 v = *reinterpret_cast<const u32x4_a4*>(row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = c + i < cols ? load1(row + c + i) : 0.f;
    }
}

template <class T, int V>
__global__ void __launch_bounds__(kMaxWaves* kWaveSize)
ln_backward_few_kernel(LnBwd p, int row_blocks, float* dw_out, float* db_out) {
    __shared__ float4 s_dw[kMaxWaves * 4][16], s_db[kMaxWaves * 4][16];
    if ((int)blockIdx.x < row_blocks) {
        const int tw = p.waves * kWaveSize;
        const Share<V> c((int)threadIdx.x % tw, tw, (int)p.cols);
        float dw[V][8], db[V][8], dwt, dbt;   // (not touched)
        backward_rows<T, V, false, kStreamNone>(p, c, blockIdx.x, row_blocks, dw, db, dwt, dbt);
        return;
    }
    const int cx = threadIdx.x % 16, slice = threadIdx.x / 16, slices = blockDim.x / 16;
    const int64_t c0 = (int64_t)((int)blockIdx.x - row_blocks) * 64;
    const int64_t c = c0 + cx * 4;
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    float dw[4] = {0.f, 0.f, 0.f, 0.f}, db[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int r = slice; r < (int)p.rows; r += slices) {
        float fx[4], fd[4];
        load4(x + r * p.cols, c, p.cols, fx);
        load4(dy + r * p.cols, c, p.cols, fd);
        const float mean = p.mean[r], rstd = p.rstd[r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            dw[i] = fmaf(fd[i], (fx[i] - mean) * rstd, dw[i]);
            db[i] += fd[i];
        }
    }
    s_dw[slice][cx] = float4{dw[0], dw[1], dw[2], dw[3]};
    s_db[slice][cx] = float4{db[0], db[1], db[2], db[3]};
    __syncthreads();
    const int col = threadIdx.x % 64;
    if (threadIdx.x >= 128 || c0 + col >= p.cols) return;
    const float* src = reinterpret_cast<const float*>(threadIdx.x < 64 ? s_dw[0] : s_db[0]) + col;
    float sum = 0.f;
    for (int i = 0; i < slices; ++i) sum += src[i * 64];
    (threadIdx.x < 64 ? dw_out : db_out)[c0 + col] = sum;
}

// Long rows: dx, one workgroup per row, swept twice (bound as the forward's:
// 4096 x 32768 bf16 with a residual 260 us).
template <class T>
__global__ void __launch_bounds__(kLongThreads)
ln_backward_long_kernel(LnBwd p) {
    __shared__ float red[kMaxWaves];
    for (int64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        const T* xr = static_cast<const T*>(p.x) + r * p.cols;
        const T* dyr = static_cast<const T*>(p.dy) + r * p.cols;
        const T* rr = p.res ? static_cast<const T*>(p.res) + r * p.cols : nullptr;
        T* dxr = static_cast<T*>(p.dx) + r * p.cols;
        const float mean = p.mean[r], rstd = p.rstd[r];
        float s1 = 0.f, s2 = 0.f;
        auto add = [&](float x, float d, float w) {
            s1 = fmaf(d, w, s1);
            s2 = fmaf(d * w, (x - mean) * rstd, s2);
        };
        for_columns(p.cols,
                    [&](int64_t c) {
                        Raw8<T> vx, vd;
                        float w[8];
                        vx.load(xr + c);
                        vd.load(dyr + c);
                        load_param8(p.w, p.param_bf16, c, 1.f, w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) add(vx.get(i), vd.get(i), w[i]);
                    },
                    [&](int64_t c) {
                        add(load1(xr + c), load1(dyr + c), load_param1(p.w, p.param_bf16, c, 1.f));
                    });
        const float c1 = block_sum(s1, red) / (float)p.cols;
        const float c2 = block_sum(s2, red) / (float)p.cols;
        auto out = [&](float x, float d, float w, float res) {
            return fmaf(rstd, d * w - c1 - (x - mean) * rstd * c2, res);
        };
        for_columns(p.cols,
                    [&](int64_t c) {
                        Raw8<T> vx, vd, vr;
                        float w[8], f[8];
                        vx.load(xr + c);
                        vd.load(dyr + c);
                        if (rr) vr.load(rr + c); else vr.zero();
                        load_param8(p.w, p.param_bf16, c, 1.f, w);
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = out(vx.get(i), vd.get(i), w[i], vr.get(i));
                        store8(dxr + c, f);
                    },
                    [&](int64_t c) {
                        store1(dxr + c, out(load1(xr + c), load1(dyr + c),
                                            load_param1(p.w, p.param_bf16, c, 1.f), rr ? load1(rr + c) : 0.f));
                    });
    }
}

// Long rows: partial column sums.  Workgroup (part, column block): 256 columns,
// one per thread, over the rows part, part + parts, ... (4096 x 32768 bf16 168 us,
// 3.2 TB/s: two bytes a lane).
constexpr int kColThreads = 256;

template <class T>
__global__ void __launch_bounds__(kColThreads)
ln_column_sums_kernel(LnBwd p, int parts) {
    const int64_t c = (int64_t)blockIdx.x * kColThreads + threadIdx.x;
    const int part = blockIdx.y;
    if (c >= p.cols) return;
    const T* x = static_cast<const T*>(p.x);
    const T* dy = static_cast<const T*>(p.dy);
    float dw = 0.f, db = 0.f;
    for (int64_t r = part; r < p.rows; r += parts) {
        const float d = load1(dy + r * p.cols + c);
        dw = fmaf(d, (load1(x + r * p.cols + c) - p.mean[r]) * p.rstd[r], dw);
        db += d;
    }
    p.partial[part * p.pitch + c] = dw;
    p.partial[(parts + part) * p.pitch + c] = db;
}

// dw and db from the partial rows (blockIdx.y 0: dw, 1: db).  A workgroup takes
// 64 columns: 16 lanes of 4 columns each, 32 slices of the parts (8 of 256 parts,
// all loaded before the first is added), joined in a fixed order: 256 parts of
// 8192 columns 5.0 us (17 MB), of 1000 3.9 us.  parts == 0
// (no rows) gives zeros.
constexpr int kReduceSlices = 32;

__global__ void __launch_bounds__(kReduceSlices * 16)
ln_reduce_kernel(const float* partial, int parts, int64_t pitch, int64_t cols, float* dw, float* db) {
    __shared__ float4 s[kReduceSlices][16];
    const int cx = threadIdx.x % 16, slice = threadIdx.x / 16;
    const int64_t c = (int64_t)blockIdx.x * 64 + cx * 4;
    const float* src = partial + (int64_t)blockIdx.y * parts * pitch;
    float4 a{0.f, 0.f, 0.f, 0.f};
    for (int i0 = slice; i0 < parts; i0 += 8 * kReduceSlices) {   // (the pitch covers whole 64-column blocks)
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int i = i0 + k * kReduceSlices;
            v[k] = i < parts ? *reinterpret_cast<const float4*>(src + i * pitch + c) : float4{0.f, 0.f, 0.f, 0.f};
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            a.x += v[k].x;
            a.y += v[k].y;
            a.z += v[k].z;
            a.w += v[k].w;
        }
    }
    s[slice][cx] = a;
    __syncthreads();
    if (threadIdx.x < 64) {
        const int64_t col = (int64_t)blockIdx.x * 64 + threadIdx.x;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kReduceSlices; ++i) sum += reinterpret_cast<const float*>(s[i])[threadIdx.x];
        if (col < cols) (blockIdx.y ? db : dw)[col] = sum;
    }
}

// ---------------------------------------------------------------- host ---

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t min64(int64_t a, int64_t b) { return a < b ? a : b; }
int64_t max64(int64_t a, int64_t b) { return a > b ? a : b; }

int device_cu_count() {
    int dev = -1, cus = 0;
    if (hipGetDevice(&dev) != hipSuccess) return 0;
    if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess) return 0;
    return cus;
}

bool aligned_to(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_shape(int64_t rows, int64_t cols) {
    if (rows < 0 || rows > INT32_MAX || cols < 1 || cols > (int64_t(1) << 24)) return FP8LN_ERR_SHAPE;
    return FP8LN_OK;
}

int row_waves(int64_t cols, int vecs) { return (int)max64(1, ceil_div(cols / 8, kWaveSize * vecs)); }

// How the gradient's rows are shared out.  It does not depend on the device:
// the sums' order has to be the same on every one.
constexpr int64_t kGradWorkgroups = 256;
constexpr int64_t kLongParts = 64;
struct GradPlan {
    bool held, few;
    int vecs, waves, subs;
    int64_t parts, pitch;
};

// Few rows: one launch that reads dy and x twice beats partial sums (MI355X,
// bf16 / fp32 with a residual, one launch against two: 64 x 8192 3.9 / 5.2 us
// against 8.6 / 9.1, 128 x 1000 5.0 / 5.2 against 5.9 / 5.7, 512 x 4096 7.6 / 10.7
// against 12.2 / 13.7) until each workgroup's columns are too long a walk
// (512 x 1000 7.3 / 7.5 against 7.2 / 7.1, 1024 x 8192 21.7 / 26.1 against 19.9 / 22.8).
bool few_rows(int64_t rows, int64_t cols) { return rows <= min64(768, 256 + cols / 8); }

GradPlan grad_plan(int64_t rows, int64_t cols, int dtype) {
    GradPlan g;
    g.held = cols <= kHeldCols;
    g.few = g.held && few_rows(rows, cols);
    g.pitch = ceil_div(cols, 64) * 64;
    g.vecs = kVecs;
    if (!g.held) {
        g.waves = g.subs = 0;
        g.parts = min64(rows, kLongParts);
        return g;
    }
    // fp32 rows take one vector a lane where 16 waves reach (two would spill).
    if (dtype == FP8LN_FP32 && cols / 8 <= kMaxWaves * kWaveSize) g.vecs = 1;
    g.waves = row_waves(cols, g.vecs);
    if (g.few) {
        // A column workgroup has 4 slices of rows for each wave: about 4 rows each.
        g.subs = (int)max64(1, min64(kMaxWaves, max64(4, rows / 16)) / g.waves);
        g.parts = 0;
        return g;
    }
    g.subs = (int)max64(1, min64(kMaxWaves / g.waves, ceil_div(rows, kGradWorkgroups)));
    g.parts = min64(kGradWorkgroups, ceil_div(rows, g.subs));
    return g;
}

// Partial results: the most that either element type takes.
int64_t grad_workspace(int64_t rows, int64_t cols) {
    const int64_t pitch = ceil_div(cols, 64) * 64;
    return 2 * min64(rows, cols <= kHeldCols ? kGradWorkgroups : kLongParts) * pitch * (int64_t)sizeof(float);
}

template <bool WIDE>
void launch_forward(const LnFwd& p, int dtype, dim3 grid, dim3 block, hipStream_t hs) {
    const int64_t bytes = p.rows * p.cols * (2 + (p.y ? 2 : 0) + (p.q ? 1 : 0));   // (bf16)
    if (dtype == FP8LN_FP32) hipLaunchKernelGGL((ln_forward_kernel<float, WIDE, false>), grid, block, 0, hs, p);
    else if (bytes > kCachedBytes) hipLaunchKernelGGL((ln_forward_kernel<bf16_t, WIDE, true>), grid, block, 0, hs, p);
    else hipLaunchKernelGGL((ln_forward_kernel<bf16_t, WIDE, false>), grid, block, 0, hs, p);
}

template <class T, int V>
void launch_backward(const LnBwd& p, const GradPlan& g, float* dw, float* db, hipStream_t hs) {
    const dim3 block(g.waves * g.subs * kWaveSize);
    if (g.few) {
        const int row_blocks = (int)ceil_div(p.rows, g.subs);
        hipLaunchKernelGGL((ln_backward_few_kernel<T, V>), dim3((unsigned)(row_blocks + ceil_div(p.cols, 64))), block,
                           0, hs, p, row_blocks, dw, db);
        return;
    }
    const unsigned lds = (unsigned)(g.subs / 2 * 4 * V * g.waves * kWaveSize * sizeof(float4));
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3((unsigned)g.parts), block, lds, hs, p); };
    if constexpr (std::is_same_v<T, bf16_t>) {
        // dx too where a row is long (16384 x 8192 183 us against 198 with the
        // hint on the loads alone, 32768 x 2048 77 against 74).
        if (p.rows * p.cols * (p.res ? 4 : 3) * (int64_t)sizeof(T) > kCachedBytes)
            return p.cols >= 4096 ? go(ln_backward_kernel<T, V, kStreamAll>) : go(ln_backward_kernel<T, V, kStreamLoads>);
    }
    go(ln_backward_kernel<T, V, kStreamNone>);
}

}  // namespace

extern "C" {

int fp8_layer_norm(const void* x, int dtype, const void* w, const void* b, int param_dtype, float eps,
                   void* y, void* q, int q_format, float* scale, float* mean, float* rstd,
                   int64_t rows, int64_t cols, struct ihipStream_t* stream) {
    if ((dtype != FP8LN_BF16 && dtype != FP8LN_FP32) || (param_dtype != FP8LN_BF16 && param_dtype != FP8LN_FP32))
        return FP8LN_ERR_DTYPE;
    if (q && q_format != FP8LN_E4M3FN && q_format != FP8LN_E5M2) return FP8LN_ERR_DTYPE;
    const int st = check_shape(rows, cols);
    if (st != FP8LN_OK) return st;
    if (q && cols % 16 != 0) return FP8LN_ERR_SHAPE;
    if (!(eps >= 0.f) || std::isinf(eps)) return FP8LN_ERR_VALUE;
    if (rows == 0) return FP8LN_OK;
    if (!x || (!y && !q) || !q != !scale || !mean != !rstd) return FP8LN_ERR_NULL;
    const uintptr_t ea = dtype == FP8LN_BF16 ? 2 : 4, pa = param_dtype == FP8LN_BF16 ? 2 : 4;
    if (!aligned_to(x, ea) || !aligned_to(y, ea) || !aligned_to(w, pa) || !aligned_to(b, pa) ||
        !aligned_to(q, 16) || !aligned_to(scale, 4) || !aligned_to(mean, 4) || !aligned_to(rstd, 4))
        return FP8LN_ERR_ALIGN;
    const int cus = device_cu_count();
    if (cus <= 0) return FP8LN_ERR_DEVICE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    LnFwd p{x, w, b, param_dtype == FP8LN_BF16, eps, y, static_cast<uint8_t*>(q), q_format, scale, mean, rstd,
            rows, cols, row_waves(cols, kVecs)};
    (void)hipGetLastError();
    if (cols > kHeldCols) {
        const dim3 grid((unsigned)min64(rows, (int64_t)cus * 8));
        if (dtype == FP8LN_BF16)
            hipLaunchKernelGGL(ln_forward_long_kernel<bf16_t>, grid, dim3(kLongThreads), 0, hs, p);
        else
            hipLaunchKernelGGL(ln_forward_long_kernel<float>, grid, dim3(kLongThreads), 0, hs, p);
    } else if (p.waves == 1) {
        constexpr int kRows = 4;   // waves, and so rows, per workgroup
        const dim3 grid((unsigned)min64(ceil_div(rows, kRows), (int64_t)cus * 4));
        launch_forward<false>(p, dtype, grid, dim3(kRows * kWaveSize), hs);
    } else {
        const dim3 grid((unsigned)min64(rows, (int64_t)cus * (kMaxWaves / p.waves)));
        launch_forward<true>(p, dtype, grid, dim3(p.waves * kWaveSize), hs);
    }
    if (hipGetLastError() != hipSuccess) return FP8LN_ERR_LAUNCH;
    return FP8LN_OK;
}

int64_t fp8_layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
    if (check_shape(rows, cols) != FP8LN_OK || rows == 0) return 0;
    return grad_workspace(rows, cols);
}

int fp8_layer_norm_backward(const void* dy, const void* x, int dtype, const float* mean,
                            const float* rstd, const void* w, int param_dtype,
                            const void* residual_grad, void* dx, float* dw, float* db, int64_t rows,
                            int64_t cols, void* workspace, int64_t workspace_bytes,
                            struct ihipStream_t* stream) {
    if ((dtype != FP8LN_BF16 && dtype != FP8LN_FP32) || (param_dtype != FP8LN_BF16 && param_dtype != FP8LN_FP32))
        return FP8LN_ERR_DTYPE;
    const int st = check_shape(rows, cols);
    if (st != FP8LN_OK) return st;
    if (!dw || !db || (rows > 0 && (!dy || !x || !mean || !rstd || !dx))) return FP8LN_ERR_NULL;
    const uintptr_t ea = dtype == FP8LN_BF16 ? 2 : 4, pa = param_dtype == FP8LN_BF16 ? 2 : 4;
    if (!aligned_to(dy, ea) || !aligned_to(x, ea) || !aligned_to(residual_grad, ea) || !aligned_to(dx, ea) ||
        !aligned_to(w, pa) || !aligned_to(mean, 4) || !aligned_to(rstd, 4) || !aligned_to(dw, 4) ||
        !aligned_to(db, 4))
        return FP8LN_ERR_ALIGN;
    if (rows > 0 && (!workspace || workspace_bytes < grad_workspace(rows, cols))) return FP8LN_ERR_WORKSPACE;
    if (rows > 0 && !aligned_to(workspace, 256)) return FP8LN_ERR_ALIGN;
    const int cus = device_cu_count();
    if (cus <= 0) return FP8LN_ERR_DEVICE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const GradPlan g = grad_plan(rows, cols, dtype);
    LnBwd p{dy, x, mean, rstd, w, param_dtype == FP8LN_BF16, residual_grad, dx, static_cast<float*>(workspace),
            rows, cols, g.pitch, g.waves, g.subs};
    std::lock_guard<std::mutex> together(fp8mm::enqueue_lock(workspace));
    (void)hipGetLastError();
    if (rows > 0 && g.held) {
        if (dtype == FP8LN_BF16) launch_backward<bf16_t, 2>(p, g, dw, db, hs);
        else if (g.vecs == 1) launch_backward<float, 1>(p, g, dw, db, hs);
        else launch_backward<float, 2>(p, g, dw, db, hs);
    } else if (rows > 0) {
        const dim3 grid((unsigned)min64(rows, (int64_t)cus * 8));
        const dim3 cgrid((unsigned)ceil_div(cols, kColThreads), (unsigned)g.parts);
        if (dtype == FP8LN_BF16) {
            hipLaunchKernelGGL(ln_column_sums_kernel<bf16_t>, cgrid, dim3(kColThreads), 0, hs, p, (int)g.parts);
            hipLaunchKernelGGL(ln_backward_long_kernel<bf16_t>, grid, dim3(kLongThreads), 0, hs, p);
        } else {
            hipLaunchKernelGGL(ln_column_sums_kernel<float>, cgrid, dim3(kColThreads), 0, hs, p, (int)g.parts);
            hipLaunchKernelGGL(ln_backward_long_kernel<float>, grid, dim3(kLongThreads), 0, hs, p);
        }
    }
    if (rows == 0 || !g.few)
        hipLaunchKernelGGL(ln_reduce_kernel, dim3((unsigned)ceil_div(cols, 64), 2), dim3(kReduceSlices * 16), 0, hs,
                           static_cast<const float*>(workspace), (int)g.parts, g.pitch, cols, dw, db);
    if (hipGetLastError() != hipSuccess) return FP8LN_ERR_LAUNCH;
    return FP8LN_OK;
}

const char* fp8_layer_norm_status_string(int s) {
    switch (s) {
        case FP8LN_OK: return "ok";
        case FP8LN_ERR_NULL: return "a required pointer is NULL (q comes with scale, mean with rstd)";
        case FP8LN_ERR_SHAPE:
            return "rows or cols out of range (need 0<=rows<2^31, 1<=cols<=2^24, cols%16==0 for codes)";
        case FP8LN_ERR_ALIGN:
            return "misaligned pointer (tensors: their element; q: 16 B; workspace: 256 B)";
        case FP8LN_ERR_DTYPE: return "unknown element type or code format";
        case FP8LN_ERR_DEVICE: return "no usable HIP device";
        case FP8LN_ERR_LAUNCH: return "kernel launch failed";
        case FP8LN_ERR_WORKSPACE:
            return "workspace smaller than fp8_layer_norm_backward_workspace_size()";
        case FP8LN_ERR_VALUE: return "eps must be finite and not negative";
        default: return "unknown status";
    }
}

}  // extern "C"
