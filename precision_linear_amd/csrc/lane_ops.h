// Loads, stores and lane exchanges shared by the memory-bound kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "fp8_convert.h"

namespace {

constexpr int kWaveSize = 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x4 u32x4_a2 __attribute__((aligned(2)));
typedef u32x4 u32x4_a4 __attribute__((aligned(4)));

typedef uint16_t bf16_t;

// ------------------------------------------------------------ elements ---

// Memory that a launch reads or writes once, more of it than the 256 MB of the
// memory-side cache: with the non-temporal hint (NT) it does not push out of the
// L2 what the launch still needs, or what it has yet to write back whole.
constexpr int64_t kCachedBytes = int64_t(256) << 20;
template <bool NT, class V, class P>
__device__ __forceinline__ V load_hinted(const P* p) {
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool NT, class V, class P>
__device__ __forceinline__ void store_hinted(P* p, V v) {
    if constexpr (NT) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// 8 consecutive elements as they lie in memory.
template <class T> struct Raw8;
template <> struct Raw8<bf16_t> {
    u32x4 v;
    template <bool NT = false>
    __device__ __forceinline__ void load(const bf16_t* p) {
        v = load_hinted<NT, u32x4>(reinterpret_cast<const u32x4_a2*>(p));
    }
    __device__ __forceinline__ void zero() { v = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ float get(int i) const {
        const uint32_t w = v[i / 2];
        return i % 2 ? bf16_hi(w) : bf16_lo(w);
    }
};
template <> struct Raw8<float> {
    u32x4 v[2];
    template <bool NT = false>
    __device__ __forceinline__ void load(const float* p) {
        static_assert(!NT, "a lane's two halves share lines with its neighbours': the hint would drop them half used");
        v[0] = *reinterpret_cast<const u32x4_a4*>(p);
        v[1] = *reinterpret_cast<const u32x4_a4*>(p + 4);
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = u32x4{0u, 0u, 0u, 0u}; }
    __device__ __forceinline__ float get(int i) const { return __uint_as_float(v[i / 4][i % 4]); }
};

__device__ __forceinline__ float load1(const bf16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// fp32 -> bf16, round to nearest even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    typedef float f2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{lo, hi}, bf2));
}

template <bool NT = false>
__device__ __forceinline__ void store8(bf16_t* p, const float (&f)[8]) {
    store_hinted<NT>(reinterpret_cast<u32x4_a2*>(p), u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                           pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])});
}
template <bool NT = false>
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
    static_assert(!NT, "as for the loads");
#pragma unroll
    for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u32x4_a4*>(p + 4 * h) =
            u32x4{__float_as_uint(f[4 * h]), __float_as_uint(f[4 * h + 1]), __float_as_uint(f[4 * h + 2]),
                  __float_as_uint(f[4 * h + 3])};
}
__device__ __forceinline__ void store1(bf16_t* p, float f) { *p = (bf16_t)pack_bf16(f, f); }
__device__ __forceinline__ void store1(float* p, float f) { *p = f; }

// ----------------------------------------------------------- reductions ---

// Lane exchanges inside a row of 16 lanes (DPP: no LDS round trip).
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
constexpr int kSwap1 = 0xB1;         // quad_perm [1, 0, 3, 2]
constexpr int kSwap2 = 0x4E;         // quad_perm [2, 3, 0, 1]
constexpr int kHalfMirror = 0x141;   // lane i of 8 reads lane 7 - i
constexpr int kMirror = 0x140;       // lane i of 16 reads lane 15 - i

__device__ __forceinline__ float lane_value(float x, int lane) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), lane));
}

// Sum over each row of 16 lanes, in every lane of it.
__device__ __forceinline__ float row16_sum(float x) {
    x += dpp<kSwap1>(x);
    x += dpp<kSwap2>(x);
    x += dpp<kHalfMirror>(x);
    return x + dpp<kMirror>(x);
}
__device__ __forceinline__ float row16_max(float x) {
    x = fmaxf(x, dpp<kSwap1>(x));
    x = fmaxf(x, dpp<kSwap2>(x));
    x = fmaxf(x, dpp<kHalfMirror>(x));
    return fmaxf(x, dpp<kMirror>(x));
}
// Over the wave; every lane active, every lane returns the same.
__device__ __forceinline__ float wave_sum(float x) {
    x = row16_sum(x);
    return (lane_value(x, 0) + lane_value(x, 16)) + (lane_value(x, 32) + lane_value(x, 48));
}
__device__ __forceinline__ float wave_max(float x) {
    x = row16_max(x);
    return fmaxf(fmaxf(lane_value(x, 0), lane_value(x, 16)), fmaxf(lane_value(x, 32), lane_value(x, 48)));
}

}  // namespace
