// The AdamW step over many tensors for gfx950 (MI355X) (formulas and the random
// rounding: include/adamw.h).
//
// Bound by memory: with fp32 moments, an fp32 parameter and a bf16 gradient an element
// is 14 bytes read and 12 written; with 8-bit moments 8 and 6.  The tensors' addresses go
// into the kernel's arguments (48 tensors a launch), so nothing is copied to the GPU
// beforehand and a capture holds them.  A workgroup takes a chunk of one tensor, which it
// finds by the first chunks of all; a wave takes 256 elements, a block of the 8-bit
// moments, at a time, with several of them in flight.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>
#include <utility>
#include <vector>

#include "../../include/adamw.h"
#include "lane_ops.h"

namespace {

constexpr int kTensors = 48;              // of a launch (the arguments stay under 4 KiB)
constexpr int kBlock = 256;               // elements of a block and of a wave at a time
constexpr int kStepThreads = 256;
constexpr int kWaves = kStepThreads / kWaveSize;

// Blocks of a wave in flight: loads enough, and registers few enough for more waves (us on
// one MI355X of 2, 3 and 4: 4.7e8 elements with fp32 moments 2196, 2202 and 2128, with 8-bit
// ones 1143, 1152 and 1171; 1.1e8 with a master 524, 533 and 561).
constexpr int in_flight(int bits, bool master) { return bits == 8 || master ? 2 : 4; }
constexpr int chunk_size(int bits, bool master) { return kBlock * kWaves * in_flight(bits, master); }

struct Entry {
    void* param;
    const void* grad;
    void* m;
    void* v;
    float* master;
    float* m_scale;
    float* v_scale;
    int64_t numel;
    int64_t first_block;                  // blocks of the call's tensors before this one
};

struct StepArgs {
    Entry t[kTensors];
    uint32_t first_chunk[kTensors];
    int count;
    float beta1, beta1_rest, beta2, beta2_rest, eps;
    float lr, weight_decay;
    float corr1, corr2;                   // 1 / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
    uint32_t seed;
    double log_beta1, log_beta2;
    const float* lr_ptr;
    const float* step_ptr;
    const int64_t* seed_ptr;
    const float* grad_scale_ptr;
};
static_assert(sizeof(StepArgs) <= 4096, "kernel arguments");

// Four elements as they lie in memory, at any address that suits one.
template <class T> struct Raw4;
template <> struct Raw4<float> {
    u32x4 v;
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i]); }
    __device__ __forceinline__ void set(const float (&f)[4]) {
        v = u32x4{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])};
    }
    typedef u32x4_a4 memory;
};
template <> struct Raw4<bf16_t> {
    u32x2 v;
    __device__ __forceinline__ float get(int i) const { return i % 2 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]); }
    __device__ __forceinline__ void set(const float (&f)[4]) { v = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])}; }
    typedef u32x2 memory __attribute__((aligned(2)));
};
template <> struct Raw4<uint8_t> {        // e4m3fn
    uint32_t v;
    __device__ __forceinline__ float get(int i) const {
        return i == 0   ? __builtin_amdgcn_cvt_f32_fp8((int)v, 0)
               : i == 1 ? __builtin_amdgcn_cvt_f32_fp8((int)v, 1)
               : i == 2 ? __builtin_amdgcn_cvt_f32_fp8((int)v, 2)
                        : __builtin_amdgcn_cvt_f32_fp8((int)v, 3);
    }
    __device__ __forceinline__ void set(const float (&f)[4]) {
        const int w = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], 0, false);
        v = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], w, true);
    }
    typedef uint32_t memory __attribute__((aligned(1)));
};

// The elements from `at` on, `left` of them (4 or more: all).
template <bool NT, class T>
__device__ __forceinline__ Raw4<T> load4(const T* p, int64_t at, int64_t left) {
    Raw4<T> r;
    if (left >= 4) {
        const auto* from = reinterpret_cast<const typename Raw4<T>::memory*>(p + at);
        if constexpr (NT) r.v = __builtin_nontemporal_load(from);
        else r.v = *from;
    } else {
        T e[4] = {};
        for (int i = 0; i < left; ++i) e[i] = p[at + i];
        __builtin_memcpy(&r.v, e, sizeof(e));
    }
    return r;
}
template <bool NT, class T>
__device__ __forceinline__ void store4(T* p, int64_t at, int64_t left, const float (&f)[4]) {
    Raw4<T> r;
    r.set(f);
    if (left >= 4) {
        auto* to = reinterpret_cast<typename Raw4<T>::memory*>(p + at);
        if constexpr (NT) __builtin_nontemporal_store(r.v, to);
        else *to = r.v;
    } else {
        T e[4];
        __builtin_memcpy(e, &r.v, sizeof(e));
        for (int i = 0; i < left; ++i) p[at + i] = e[i];
    }
}

// 32 random bits of the i-th position from the one whose h0 is `start`.
__device__ __forceinline__ uint32_t random_bits(uint32_t start, uint32_t i) {
    uint32_t h = start + i * 0x6A09E667u;
    h = (h ^ (h >> 15)) * 0x3C6EF373u;
    h = (h ^ (h >> 13)) * 0xA54FF53Bu;
    return h ^ (h >> 16);
}

// y, |y| <= 448 up to a rounding or two, to one of its neighbours in e4m3fn: up (in
// magnitude) where the part of a step that is left and r / 2^16 make one (r4 is r 2^4; the
// last bits of a y that rounding has put above 448 are too few for that).  Below 2^-6
// the steps are those of 2^-6, so that is added meanwhile.  NaN stays NaN: the addition
// saturates.
template <bool POSITIVE>
__device__ __forceinline__ float round_at_random(float y, int r4) {
    float t = fabsf(y);
    const float lift = t < 0x1p-6f ? 0x1p-6f : 0.f;
    t = __int_as_float(__builtin_elementwise_add_sat(__float_as_int(t + lift), r4) & (int)0xfff00000) - lift;
    if (POSITIVE) return y > 0.f && t == 0.f ? 0x1p-9f : t;
    return copysignf(t, y);
}

// sqrt(v), correctly rounded, for v = 0, 2^-96 and more, inf (which gives itself: the
// tests are of NaNs) and NaN.  The hardware's s is at most one step h off: v lies below the
// midpoint to its lower neighbour, (s - h / 2)^2 = s (s - h) + h^2 / 4, where v <= s (s - h), and
// above the one to the upper where v > s (s + h), h^2 / 4 being less than a last bit of v.
__device__ __forceinline__ float root_of(float v) {
    const float s = __builtin_amdgcn_sqrtf(v);
    const float down = __uint_as_float(__float_as_uint(s) - 1), up = __uint_as_float(__float_as_uint(s) + 1);
    const float by_down = fmaf(-down, s, v), by_up = fmaf(-up, s, v);
    return by_down <= 0.f ? down : by_up > 0.f ? up : s;
}
// The same of four, smaller ones too (which the hardware takes for 0): those are lifted.
__device__ __forceinline__ void roots_of(const float (&v)[4], float (&root)[4]) {
    uint32_t least = ~0u;   // (0 becomes the largest)
#pragma unroll
    for (int i = 0; i < 4; ++i) least = min(least, __float_as_uint(v[i]) - 1u);
    if (__any(least < 0x0f800000u - 1u)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) root[i] = v[i] < 0x1p-96f ? root_of(v[i] * 0x1p64f) * 0x1p-32f : root_of(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) root[i] = root_of(v[i]);
    }
}
// a / b; with 8-bit moments by the hardware's reciprocal (1 ulp), as the step would
// otherwise be bound by its arithmetic.
template <bool FAST>
__device__ __forceinline__ float quotient(float a, float b) {
    return FAST ? a * __builtin_amdgcn_rcpf(b) : a / b;
}

// The scale of a block whose largest magnitude is amax, and what values are
// multiplied by.
__device__ __forceinline__ float2 block_scale(float amax) {
    float s = amax / 448.f;
    if (s < 0x1p-100f) s = 0.f;
    return float2{s, s == 0.f ? 0.f : 1.f / s};
}

template <class P, class G, int BITS, bool MASTER, bool NT>
__global__ void __launch_bounds__(kStepThreads) adamw_kernel(StepArgs a) {
    typedef std::conditional_t<BITS == 8, uint8_t, float> S;
    typedef std::conditional_t<MASTER, float, P> W;       // what the step reads and writes
    constexpr int kInFlight = in_flight(BITS, MASTER), kChunk = chunk_size(BITS, MASTER);
    // This workgroup's tensor.
    int lo = 0, hi = a.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (a.first_chunk[mid] <= blockIdx.x) lo = mid;
        else hi = mid;
    }
    const Entry& e = a.t[lo];
    const int64_t base = (int64_t)(blockIdx.x - a.first_chunk[lo]) * kChunk;
    const int wave = threadIdx.x / kWaveSize, lane = threadIdx.x % kWaveSize;
    W* w = MASTER ? reinterpret_cast<W*>(e.master) : static_cast<W*>(e.param);
    P* param = static_cast<P*>(e.param);
    const G* grad = static_cast<const G*>(e.grad);
    S* m = static_cast<S*>(e.m);
    S* v = static_cast<S*>(e.v);

    // Blocks wave, wave + kWaves, ... of the chunk.
    int64_t at[kInFlight], left[kInFlight];
    Raw4<W> rw[kInFlight];
    Raw4<G> rg[kInFlight];
    Raw4<S> rm[kInFlight], rv[kInFlight];
    float ms[kInFlight], vs[kInFlight];
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
        at[u] = base + (u * kWaves + wave) * kBlock + lane * 4;
        left[u] = e.numel - at[u];
        rw[u] = load4<NT>(w, at[u], left[u]);
        rg[u] = load4<NT>(grad, at[u], left[u]);
        rm[u] = load4<NT>(m, at[u], left[u]);
        rv[u] = load4<NT>(v, at[u], left[u]);
        if constexpr (BITS == 8) {
            const int64_t b = at[u] / kBlock;
            const bool live = at[u] - lane * 4 < e.numel;
            ms[u] = live ? e.m_scale[b] : 0.f;
            vs[u] = live ? e.v_scale[b] : 0.f;
        }
    }
    float lr = a.lr, corr1 = a.corr1, corr2 = a.corr2;
    if (a.lr_ptr) lr = *a.lr_ptr;
    if (a.step_ptr) {
        const double t = (double)*a.step_ptr;
        corr1 = (float)(-1.0 / expm1(t * a.log_beta1));
        corr2 = (float)sqrt(-1.0 / expm1(t * a.log_beta2));
    }
    const float decay = 1.f - lr * a.weight_decay, rate = lr * corr1;
    const float gs = a.grad_scale_ptr ? *a.grad_scale_ptr : 1.f;
    const uint32_t seed = (a.seed_ptr ? (uint32_t)*a.seed_ptr : a.seed) * 0xBB67AE85u;
#pragma unroll
    for (int u = 0; u < kInFlight; ++u) {
        float fm[4], root[4], fv[4], fw[4], fg[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) fg[i] = rg[u].get(i);
        if (a.grad_scale_ptr)
#pragma unroll
            for (int i = 0; i < 4; ++i) fg[i] *= gs;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float g = fg[i];
            float m0 = rm[u].get(i), v0 = rv[u].get(i);
            if constexpr (BITS == 8) {
                m0 *= ms[u];
                v0 *= vs[u];
                v0 *= v0;
            }
            {
                // Each product and sum rounds, as the formulas are written: which code a moment of
                // 8 bits is rounded to hangs on its last bit.
#pragma clang fp contract(off)
                fm[i] = a.beta1 * m0 + a.beta1_rest * g;
                fv[i] = a.beta2 * v0 + a.beta2_rest * (g * g);
            }
        }
        roots_of(fv, root);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float step = quotient<BITS == 8>(fm[i], fmaf(root[i], corr2, a.eps));
            fw[i] = fmaf(rw[u].get(i), decay, -rate * step);
        }
        if constexpr (BITS == 8) {
            float amax_m = 0.f, amax_v = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // (zeros past the tensor's end)
                amax_m = fmaxf(amax_m, fabsf(fm[i]));
                amax_v = fmaxf(amax_v, root[i]);
            }
            const float2 sm = block_scale(wave_max(amax_m)), sv = block_scale(wave_max(amax_v));
            const uint32_t start = ((uint32_t)e.first_block * (uint32_t)kBlock + (uint32_t)at[u]) * 0x6A09E667u + seed;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t r = random_bits(start, i);
                fm[i] = round_at_random<false>(fm[i] * sm.y, (int)((r & 0xffff) << 4));
                fv[i] = round_at_random<true>(root[i] * sv.y, (int)(r >> 16 << 4));
            }
            if (lane == 0 && left[u] > 0) {
                e.m_scale[at[u] / kBlock] = sm.x;
                e.v_scale[at[u] / kBlock] = sv.x;
            }
        }
        store4<NT>(m, at[u], left[u], fm);
        store4<NT>(v, at[u], left[u], fv);
        store4<NT>(w, at[u], left[u], fw);
        if constexpr (MASTER) store4<NT>(param, at[u], left[u], fw);
    }
}

// ---------------------------------------------------------------- host ---

template <class P, class G, int BITS, bool MASTER>
void launch(const StepArgs& a, uint32_t chunks, bool stream_memory, hipStream_t hs) {
    if (stream_memory)
        hipLaunchKernelGGL((adamw_kernel<P, G, BITS, MASTER, true>), dim3(chunks), dim3(kStepThreads), 0, hs, a);
    else
        hipLaunchKernelGGL((adamw_kernel<P, G, BITS, MASTER, false>), dim3(chunks), dim3(kStepThreads), 0, hs, a);
}

typedef void (*StepLaunch)(const StepArgs&, uint32_t, bool, hipStream_t);
// [gradient][32 bits][parameter: bf16, bf16 with a master, fp32]
const StepLaunch kLaunches[2][2][3] = {
    {{launch<bf16_t, bf16_t, 8, false>, launch<bf16_t, bf16_t, 8, true>, launch<float, bf16_t, 8, false>},
     {launch<bf16_t, bf16_t, 32, false>, launch<bf16_t, bf16_t, 32, true>, launch<float, bf16_t, 32, false>}},
    {{launch<bf16_t, float, 8, false>, launch<bf16_t, float, 8, true>, launch<float, float, 8, false>},
     {launch<bf16_t, float, 32, false>, launch<bf16_t, float, 32, true>, launch<float, float, 32, false>}}};

bool at_multiple(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_numbers(const adamw_numbers& n) {
    auto ok = [](double x) { return x >= 0.0 && std::isfinite(x); };
    if (!ok(n.lr) || !ok(n.eps) || !ok(n.weight_decay) || !(n.beta1 >= 0.0 && n.beta1 < 1.0) ||
        !(n.beta2 >= 0.0 && n.beta2 < 1.0) || (!n.step_ptr && n.step < 1))
        return ADAMW_ERR_VALUE;
    if (!at_multiple(n.lr_ptr, 4) || !at_multiple(n.step_ptr, 4) || !at_multiple(n.seed_ptr, 8) ||
        !at_multiple(n.grad_scale_ptr, 4))
        return ADAMW_ERR_ALIGN;
    return ADAMW_OK;
}

// Addresses [from, to) that a step writes.
struct Range {
    uintptr_t from, to;
};
bool from_less(const Range& a, const Range& b) { return a.from < b.from; }
bool in_order(const std::vector<Range>& r) {   // ascending, and none into the next
    for (size_t i = 1; i < r.size(); ++i)
        if (r[i].from < r[i - 1].to) return false;
    return true;
}

// Byte by byte from the lowest on, without branches that hang on the order.
void by_address(std::vector<Range>& r) {
    uintptr_t differ = 0;
    for (const Range& x : r) differ |= x.from ^ r[0].from;
    std::vector<Range> next(r.size());
    for (int shift = 0; shift < 64; shift += 8) {
        if ((differ >> shift & 255) == 0) continue;
        uint32_t at[256] = {};
        for (const Range& x : r) ++at[x.from >> shift & 255];
        uint32_t sum = 0;
        for (uint32_t& c : at) sum += std::exchange(c, sum);
        for (const Range& x : r) next[at[x.from >> shift & 255]++] = x;
        r.swap(next);
    }
}

// Whether two of the ranges overlap; those of a tensor lie side by side, `kinds` of them.  A list
// seldom needs sorting, which would cost a call of many small tensors more than a launch: what one
// loop has made ascends, kind by kind, but for a few places.  (us of a call of 300 tensors up to its first launch, by
// a sort of pairs and so, on a CPU that cannot foretell its branches: with masters 22 and 6.4, with
// 8-bit moments too 41 and 7.7; shuffled 65 and 14, 100 and 17; without a check 5.)
bool overlapping(std::vector<Range>& written, size_t kinds) {
    if (in_order(written)) return false;
    constexpr size_t kRuns = 64;
    if (written.size() <= kRuns) {
        std::sort(written.begin(), written.end(), from_less);
        return !in_order(written);
    }
    std::vector<Range> runs;
    runs.reserve(kRuns + 1);
    uintptr_t end = ~uintptr_t(0);
    for (size_t k = 0; k < kinds && runs.size() <= kRuns; ++k)
        for (size_t i = k; i < written.size() && runs.size() <= kRuns; i += kinds) {
            if (written[i].from < end) runs.push_back(written[i]);
            else runs.back().to = written[i].to;
            end = written[i].to;
        }
    if (runs.size() <= kRuns) {
        std::sort(runs.begin(), runs.end(), from_less);
        if (in_order(runs)) return false;
    }
    by_address(written);
    return !in_order(written);
}

}  // namespace

extern "C" {

const char* adamw_status_string(int s) {
    switch (s) {
        case ADAMW_OK: return "ok";
        case ADAMW_ERR_NULL: return "a required pointer is NULL, or one is given that does not belong";
        case ADAMW_ERR_SHAPE: return "a negative size, or more than 2^43 elements";
        case ADAMW_ERR_ALIGN: return "a pointer is not aligned to its element";
        case ADAMW_ERR_DTYPE: return "unknown type (parameters and gradients: bf16 or fp32, moments: 8 or 32 bits), or a master of fp32 parameters";
        case ADAMW_ERR_VALUE: return "lr, betas, eps, weight_decay or step out of range";
        case ADAMW_ERR_DEVICE: return "no usable HIP device";
        case ADAMW_ERR_LAUNCH: return "kernel launch failed";
        case ADAMW_ERR_ALIAS: return "parameters or their states overlap (one is given twice)";
        default: return "unknown status";
    }
}

int adamw_step(const adamw_tensor* tensors, int64_t count, int param_dtype, int grad_dtype, int state_bits,
               const adamw_numbers* numbers, struct ihipStream_t* stream) try {
    if ((param_dtype != ADAMW_BF16 && param_dtype != ADAMW_FP32) ||
        (grad_dtype != ADAMW_BF16 && grad_dtype != ADAMW_FP32) || (state_bits != 8 && state_bits != 32))
        return ADAMW_ERR_DTYPE;
    if (!numbers || (count > 0 && !tensors)) return ADAMW_ERR_NULL;
    if (count < 0) return ADAMW_ERR_SHAPE;
    const int st = check_numbers(*numbers);
    if (st != ADAMW_OK) return st;
    const uintptr_t pa = param_dtype == ADAMW_BF16 ? 2 : 4, ga = grad_dtype == ADAMW_BF16 ? 2 : 4;
    const uintptr_t sa = state_bits == 8 ? 1 : 4;
    // (an empty tensor's pointers say nothing: torch's are all NULL)
    const adamw_tensor* first = std::find_if(tensors, tensors + count, [](const adamw_tensor& t) { return t.numel > 0; });
    const bool master = first != tensors + count && first->master != nullptr;
    if (master && param_dtype == ADAMW_FP32) return ADAMW_ERR_DTYPE;
    const size_t kinds = 3 + (master ? 1 : 0) + (state_bits == 8 ? 2 : 0);
    std::vector<Range> written;
    written.reserve((size_t)count * kinds);
    auto writes = [&](const void* p, int64_t bytes) {
        if (p) written.push_back(Range{(uintptr_t)p, (uintptr_t)p + (uintptr_t)bytes});
    };
    int64_t total = 0;
    for (int64_t i = 0; i < count; ++i) {
        const adamw_tensor& t = tensors[i];
        if (t.numel < 0 || t.numel > (int64_t(1) << 43) - total) return ADAMW_ERR_SHAPE;
        total += t.numel;
        if (t.numel == 0) continue;
        const bool scales = state_bits == 8;
        if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq || (t.master != nullptr) != master ||
            (t.exp_avg_scale != nullptr) != scales || (t.exp_avg_sq_scale != nullptr) != scales)
            return ADAMW_ERR_NULL;
        if (!at_multiple(t.param, pa) || !at_multiple(t.grad, ga) || !at_multiple(t.exp_avg, sa) ||
            !at_multiple(t.exp_avg_sq, sa) || !at_multiple(t.master, 4) || !at_multiple(t.exp_avg_scale, 4) ||
            !at_multiple(t.exp_avg_sq_scale, 4))
            return ADAMW_ERR_ALIGN;
        const int64_t blocks = (t.numel + kBlock - 1) / kBlock;
        writes(t.param, t.numel * (int64_t)pa);
        writes(t.exp_avg, t.numel * (int64_t)sa);
        writes(t.exp_avg_sq, t.numel * (int64_t)sa);
        writes(t.master, t.numel * 4);
        writes(t.exp_avg_scale, blocks * 4);
        writes(t.exp_avg_sq_scale, blocks * 4);
    }
    if (overlapping(written, kinds)) return ADAMW_ERR_ALIAS;
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess) return ADAMW_ERR_DEVICE;
    const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const int64_t chunk = chunk_size(state_bits, master);
    const int64_t bytes = total * (int64_t)((master ? 10 : 2 * pa) + ga + (state_bits == 8 ? 4 : 16));
    StepArgs a;
    a.beta1 = (float)numbers->beta1;
    a.beta1_rest = (float)(1.0 - numbers->beta1);
    a.beta2 = (float)numbers->beta2;
    a.beta2_rest = (float)(1.0 - numbers->beta2);
    // An eps that is more than 0 stays so, and its reciprocal a number: 0 over it is 0.
    a.eps = numbers->eps > 0.0 ? std::max((float)numbers->eps, state_bits == 8 ? 0x1p-126f : 0x1p-149f) : 0.f;
    a.lr = (float)numbers->lr;
    a.weight_decay = (float)numbers->weight_decay;
    a.log_beta1 = log(numbers->beta1);
    a.log_beta2 = log(numbers->beta2);
    const double step = numbers->step_ptr ? 1.0 : (double)numbers->step;
    a.corr1 = (float)(-1.0 / expm1(step * a.log_beta1));
    a.corr2 = (float)sqrt(-1.0 / expm1(step * a.log_beta2));
    a.seed = numbers->seed;
    a.lr_ptr = numbers->lr_ptr;
    a.step_ptr = numbers->step_ptr;
    a.seed_ptr = numbers->seed_ptr;
    a.grad_scale_ptr = numbers->grad_scale_ptr;
    const StepLaunch run = kLaunches[grad_dtype][state_bits == 32][param_dtype == ADAMW_FP32 ? 2 : master];
    (void)hipGetLastError();
    // A launch takes up to kTensors tensors and kMaxChunks chunks; a larger tensor is
    // cut at whole blocks.
    constexpr int64_t kMaxChunks = int64_t(1) << 22;
    int64_t block = 0, chunks = 0;
    a.count = 0;
    auto flush = [&]() {
        if (a.count > 0) run(a, (uint32_t)chunks, bytes > kCachedBytes, hs);
        a.count = 0;
        chunks = 0;
    };
    for (int64_t i = 0; i < count; ++i) {
        const adamw_tensor& t = tensors[i];
        for (int64_t done = 0; done < t.numel;) {
            const int64_t n = std::min(t.numel - done, (kMaxChunks - chunks) * chunk);
            Entry& e = a.t[a.count];
            auto step_on = [&](auto* p, int64_t size) {
                return p ? (decltype(p))((uintptr_t)p + (uintptr_t)(done * size)) : p;
            };
            e.param = step_on(t.param, pa);
            e.grad = step_on(t.grad, ga);
            e.m = step_on(t.exp_avg, sa);
            e.v = step_on(t.exp_avg_sq, sa);
            e.master = step_on(t.master, 4);
            e.m_scale = t.exp_avg_scale ? t.exp_avg_scale + done / kBlock : nullptr;
            e.v_scale = t.exp_avg_sq_scale ? t.exp_avg_sq_scale + done / kBlock : nullptr;
            e.numel = n;
            e.first_block = block;
            a.first_chunk[a.count++] = (uint32_t)chunks;
            chunks += (n + chunk - 1) / chunk;
            block += (n + kBlock - 1) / kBlock;
            done += n;
            if (a.count == kTensors || chunks == kMaxChunks) flush();
        }
    }
    flush();
    return hipGetLastError() == hipSuccess ? ADAMW_OK : ADAMW_ERR_LAUNCH;
} catch (...) {
    return ADAMW_ERR_SHAPE;   // (no host memory for the list)
}

}  // extern "C"
