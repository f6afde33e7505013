// The activations of the linear layer and their slopes, in fp32.
//
//   none       z
//   relu       max(z, 0), slope 1 for z > 0 else 0
//   gelu       z Phi(z), Phi the normal distribution function
//   gelu_tanh  0.5 z (1 + tanh(u)) = z sigmoid(2 u),  u = sqrt(2/pi) (z + 0.044715 z^3)
//   silu       z sigmoid(z)
//
// Phi.  With t = |z|, Q(t) = 1 - Phi(t) = exp(-t^2 / 2) R(t), and R (smooth,
// from 1/2 down like 1 / (t sqrt(2 pi))) is s P(s) for s = 1 / (1 + p t) and a
// polynomial P.  p and P's coefficients were fitted here (weighted least
// squares, reweighted towards the least largest relative error, over 0 <= t <=
// 14): degree 8 with p = 0.3, relative error at most 1.5e-7, so Phi keeps its
// relative accuracy in the negative tail, where 1 + erf cancels.  (A shorter fit
// would do where the rounding to bf16 follows at once, but a residual that cancels
// the activation leaves its last fp32 bits.)
//
// exp2 and the reciprocal are the hardware's (1 ulp).
#pragma once

#include <hip/hip_runtime.h>

#include <type_traits>

namespace {

enum Activation { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActSilu = 4, kActCount = 5 };

constexpr float kLog2E = 1.44269504088896341f;
constexpr float kTanhA2 = 2.f * 0.79788456080286536f;   // 2 sqrt(2 / pi)
constexpr float kTanhB = 0.044715f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;

// Q(t) exp(t^2 / 2) for t >= 0.
__device__ __forceinline__ float normal_tail(float t) {
    const float s = __builtin_amdgcn_rcpf(fmaf(0.3f, t, 1.f));
    float q = 0.03567469557679612f;
    q = fmaf(q, s, -0.15720273304111515f);
    q = fmaf(q, s, 0.20635286920959425f);
    q = fmaf(q, s, -0.053683029549290925f);
    q = fmaf(q, s, 0.12856128835779043f);
    q = fmaf(q, s, 0.09991359800531395f);
    q = fmaf(q, s, 0.12075393860757816f);
    q = fmaf(q, s, 0.11962929999040094f);
    return q * s;
}

// exp(-z^2 / 2)
__device__ __forceinline__ float bell(float z) {
    return __builtin_amdgcn_exp2f(z * z * (-0.5f * kLog2E));
}

// 1 / (1 + exp(-v)), v given times log2(e)
__device__ __forceinline__ float logistic(float v) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-v));
}

template <int ACT>
__device__ __forceinline__ float activate(float z) {
    if constexpr (ACT == kActRelu) {
        return z < 0.f ? 0.f : z;   // (NaN stays NaN)
    } else if constexpr (ACT == kActGelu) {
        const float q = normal_tail(fabsf(z)) * bell(z);
        return z * (z > 0.f ? 1.f - q : q);
    } else if constexpr (ACT == kActGeluTanh) {
        const float z2 = z * z;
        return z * logistic(z * fmaf(kTanhA2 * kTanhB * kLog2E, z2, kTanhA2 * kLog2E));
    } else if constexpr (ACT == kActSilu) {
        return z * logistic(z * kLog2E);
    } else {
        return z;
    }
}

// Beyond |z| = 16 the gelus' slopes are 0 or 1 in fp32, beyond 88 silu's; their
// terms with a factor z are bounded or left out there, so that they cannot turn
// into inf * 0.
template <int ACT>
__device__ __forceinline__ float slope(float z) {
    if constexpr (ACT == kActRelu) {
        return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    } else if constexpr (ACT == kActGelu) {
        const float e = bell(z);
        const float q = normal_tail(fabsf(z)) * e;
        const float phi = z > 0.f ? 1.f - q : q;                      // (NaN for a NaN)
        return fmaf(fminf(fmaxf(z, -16.f), 16.f) * kInvSqrt2Pi, e, phi);   // e is 0 from |z| = 16 on
    } else if constexpr (ACT == kActGeluTanh) {
        const float z2 = z * z;
        const float p = logistic(z * fmaf(kTanhA2 * kTanhB * kLog2E, z2, kTanhA2 * kLog2E));
        const float d = z * p * (1.f - p) * fmaf(3.f * kTanhA2 * kTanhB, z2, kTanhA2);
        return fabsf(z) < 16.f ? p + d : p;
    } else if constexpr (ACT == kActSilu) {
        const float p = logistic(z * kLog2E);
        return fabsf(z) < 88.f ? p * fmaf(z, 1.f - p, 1.f) : p;
    } else {
        return 1.f;
    }
}

// f(integral_constant<ACT>) for the runtime `act` (uniform over the wave).
template <class F>
__device__ __forceinline__ void with_activation(int act, F f) {
    switch (act) {
        case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
        case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
        case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
        case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
        default: f(std::integral_constant<int, kActNone>{}); break;
    }
}

}  // namespace
