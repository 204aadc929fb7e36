// Activations of the fused epilogues, and their slopes (device code).
#pragma once

#include "kernels.h"

namespace mkp {
namespace {

// Activations, branch-free on the native 2^x and reciprocal instructions.
//   sigmoid(z) = 1 / (1 + e^-z)
//   silu(x) = x sigmoid(x); the tanh form of GELU, x/2 (1 + tanh u), equals
//   x sigmoid(2u) since (1 + tanh u) / 2 = sigmoid(2u)
//   GELU, x Phi(x) = x/2 (1 + erf(x / sqrt 2)), with erf from Abramowitz &
//   Stegun, Handbook of Mathematical Functions, formula 7.1.26 (absolute
//   error <= 1.5e-7): for a >= 0, 1 - erf(a) = q(a) = P(t) e^{-a^2},
//   t = 1 / (1 + p a), P a degree-5 polynomial without constant term; so
//   1 + erf(x / sqrt 2) is q(|x| / sqrt 2) for x < 0 (no cancellation in the
//   negative tail) and 2 - q for x >= 0.
__device__ __forceinline__ float sigmoid_fast(float z) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}

__device__ __forceinline__ float gelu_erf_fast(float x) {
    const float a = fabsf(x) * 0.70710678118654752f;
    const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * a);
    float poly = 1.061405429f;
    poly = fmaf(poly, t, -1.453152027f);
    poly = fmaf(poly, t, 1.421413741f);
    poly = fmaf(poly, t, -0.284496736f);
    poly = fmaf(poly, t, 0.254829592f);
    const float q = poly * t * __builtin_amdgcn_exp2f(-1.4426950408889634f * a * a);
    return 0.5f * x * (x < 0.0f ? q : 2.0f - q);
}

template <int ACT>
__device__ __forceinline__ float act_t(float v) {
    if constexpr (ACT == ACT_RELU) return v > 0.0f ? v : 0.0f;
    if constexpr (ACT == ACT_GELU) return gelu_erf_fast(v);
    if constexpr (ACT == ACT_GELU_TANH)
        return v * sigmoid_fast(2.0f * 0.79788456080286536f * (v + 0.044715f * v * v * v));
    if constexpr (ACT == ACT_SILU) return v * sigmoid_fast(v);
    return v;
}

__device__ __forceinline__ float act_apply(int act, float v) {
    switch (act) {
        case ACT_RELU: return act_t<ACT_RELU>(v);
        case ACT_GELU: return act_t<ACT_GELU>(v);
        case ACT_GELU_TANH: return act_t<ACT_GELU_TANH>(v);
        case ACT_SILU: return act_t<ACT_SILU>(v);
        default: return v;
    }
}

// The sigmoid p of u, and 1 - p for itself: with e = 2^(-log2(e) |u|), which cannot
// overflow, one is 1 / (1 + e) and the other e / (1 + e), each good to a few units of
// itself.  (1 - p of a rounded p is off by 2^-24, which the slopes multiply by z and more:
// silu's was off by 1.0e-6 at z = 17, gelu_tanh's by 2.0e-6 at z = 5.)
struct Sigmoid {
    float p, rest;
    __device__ __forceinline__ explicit Sigmoid(float u) {
        const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * fabsf(u));
        const float big = __builtin_amdgcn_rcpf(1.0f + e), small = e * big;
        p = u > 0.0f ? big : small;
        rest = u > 0.0f ? small : big;
    }
};

// d act(z) / dz.  With p the sigmoid:
//   silu       p (1 + z (1 - p))
//   gelu_tanh  p + z p (1 - p) u',  p at u = 2 c (z + 0.044715 z^3), c = sqrt(2 / pi)
//   gelu       Phi(z) + z phi(z)
//   relu       1 above 0, else 0 (at 0 too)
// Absolute errors below 0.75e-7 (Phi's) and 8 units of 2^-24, roundings of values of at
// most 1.2: 5.5e-7 (measured over |z| of 0.01 to 124: gelu 2.7e-7, gelu_tanh 2.0e-7,
// silu 2.0e-7).
template <int ACT>
__device__ __forceinline__ float act_slope(float z) {
    if constexpr (ACT == ACT_RELU) return z > 0.0f ? 1.0f : z <= 0.0f ? 0.0f : z;
    if constexpr (ACT == ACT_GELU) {
        const float a = fabsf(z) * 0.70710678118654752f;
        const float t = __builtin_amdgcn_rcpf(1.0f + 0.3275911f * a);
        float poly = 1.061405429f;
        poly = fmaf(poly, t, -1.453152027f);
        poly = fmaf(poly, t, 1.421413741f);
        poly = fmaf(poly, t, -0.284496736f);
        poly = fmaf(poly, t, 0.254829592f);
        const float e = __builtin_amdgcn_exp2f(-1.4426950408889634f * a * a);
        const float q = poly * t * e;
        return fmaf(z * 0.39894228040143268f, e, 0.5f * (z < 0.0f ? q : 2.0f - q));
    }
    if constexpr (ACT == ACT_GELU_TANH) {
        const float c = 2.0f * 0.79788456080286536f, z2 = z * z;
        const Sigmoid s(c * (z + 0.044715f * z2 * z));
        const float w = s.p * s.rest;
        return w > 0.0f ? fmaf(z * w, c * fmaf(3.0f * 0.044715f, z2, 1.0f), s.p) : s.p;
    }
    if constexpr (ACT == ACT_SILU) {
        const Sigmoid s(z);
        return s.p * fmaf(z, s.rest, 1.0f);
    }
    return 1.0f;
}

}  // namespace
}  // namespace mkp
