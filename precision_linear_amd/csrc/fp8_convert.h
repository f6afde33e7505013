// Float8 conversions shared by the kernels that write float8 codes: the
// formats' parameters and the correctly rounded division by a scale.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace {

// Format parameters: FMT 0 = e4m3fn, 1 = e5m2.
template <int FMT> struct Fp8Fmt;
template <> struct Fp8Fmt<0> {
    static constexpr float kMax = 448.f;
    template <bool HI>
    __device__ static __forceinline__ int cvt_pk(float a, float b, int old) {
        return __builtin_amdgcn_cvt_pk_fp8_f32(a, b, old, HI);
    }
};
template <> struct Fp8Fmt<1> {
    static constexpr float kMax = 57344.f;
    template <bool HI>
    __device__ static __forceinline__ int cvt_pk(float a, float b, int old) {
        return __builtin_amdgcn_cvt_pk_bf8_f32(a, b, old, HI);
    }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Correctly rounded x / s for many x and one s.
//
// r = RN(1/s) (IEEE division, once).  q0 = RN(x r) is within two ulps of x/s;
// the residual e0 = x - s q0 (one fma) and q1 = RN(q0 + e0 r) bring the
// quotient within one ulp; then, with r within half an ulp of 1/s and q1
// within one ulp of x/s, the residual e1 = x - s q1 is exact and
// RN(q1 + e1 r) = RN(x/s) (P. Markstein, "Computation of elementary functions
// on the IBM RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990; the
// final step of the IA-64 division sequences).  The argument needs the
// residuals clear of the fp32 subnormal range and r finite, so the sequence
// is taken only for 2^-60 <= s <= FLT_MAX.  There, every x that can reach a
// nonzero float8 code (|x/s| >= 2^-17, half the smallest e5m2 subnormal) has
// |x| >= 2^-77 and normal residuals, so its quotient is RN(x/s) exactly;
// smaller quotients (subnormal x) may be off in the last fp32 bits but round
// to +-0 in both formats either way.  Checked exhaustively on MI355X against
// the IEEE division: every positive finite bf16 amax (s = amax / qmax) times
// every finite bf16 x with |x| <= amax, both formats: no quotient with
// |x/s| >= 2^-17 and no float8 code differs.  Elsewhere (s tiny, infinite or
// NaN) the IEEE division is used.  The residuals are formed negated,
// e = s q - x, and subtracted, q - e r: the same values (rounding is
// symmetric), but x = -0 then gives -0 where x - s q would give +0.
//
// On this path the clamp to +-qmax is not needed: |x| <= amax, so the
// correctly rounded |x/s| is at most qmax (1 + 2^-23), which the float8
// conversion rounds to qmax (checked in the same exhaustive run, against the
// clamped IEEE quotient).  A NaN input (amax skips it) stays NaN, as it does
// through the clamp of the gist's torch code.
struct Div {
    float s, r;
    bool fast;
};

__device__ __forceinline__ Div make_div(float s) {
    Div d;
    d.s = s;
    d.r = 1.f / s;
    d.fast = s >= 0x1p-60f && s <= 3.4028234663852886e38f;
    return d;
}

__device__ __forceinline__ float div_fast(float x, const Div& d) {
    float q = x * d.r;
    float e = fmaf(d.s, q, -x);
    q = fmaf(-e, d.r, q);
    e = fmaf(d.s, q, -x);
    return fmaf(-e, d.r, q);
}

template <int FMT, bool FAST>
__device__ __forceinline__ float quant1(float x, const Div& d) {
    constexpr float kMax = Fp8Fmt<FMT>::kMax;
    if constexpr (FAST) {
        return div_fast(x, d);
    } else {
        const float y = x / d.s;
        return y != y ? y : fminf(fmaxf(y, -kMax), kMax);   // NaN passes, like torch's clamp
    }
}

}  // namespace
