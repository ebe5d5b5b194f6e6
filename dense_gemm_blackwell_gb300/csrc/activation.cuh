// activation.cuh -- the activations of a gated feed-forward block and their
// slopes, in fp32.
#pragma once

#include "elem.cuh"
#include "feedforward.h"

namespace dgb {

// 1 / (1 + e^-x): 0 for a very negative x (e^-x infinite).
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + exp2_fast(-1.4426950408889634f * x)); }

constexpr float kSqrt2OverPi = 0.7978845608028654f, kTanhCubic = 0.044715f;

// silu: g / (1 + e^-g).  gelu: g Phi(g) = g erfc(-g / sqrt 2) / 2, which keeps its accuracy for negative g, where 1 + erf
// cancels.  gelu_tanh: g (1 + tanh u) / 2 = g / (1 + e^-2u), u = sqrt(2/pi) (g + 0.044715 g^3).
__device__ __forceinline__ float activate(int act, float g) {
    if (act == GATED_SILU) return g * logistic(g);
    if (act == GATED_GELU) return 0.5f * g * erfcf(-0.7071067811865476f * g);
    return g * logistic(2.f * kSqrt2OverPi * fmaf(kTanhCubic * g * g, g, g));
}

// The activation and its derivative.
__device__ __forceinline__ float2 activate_with_slope(int act, float g) {
    if (act == GATED_SILU) {
        const float p = logistic(g);
        return make_float2(g * p, p * fmaf(g, 1.f - p, 1.f));
    }
    if (act == GATED_GELU) {
        const float phi = 0.5f * erfcf(-0.7071067811865476f * g);
        // g e^(-g^2/2) / sqrt(2 pi)
        return make_float2(g * phi, fmaf(g * 0.3989422804014327f, exp2_fast(-0.7213475204444817f * g * g), phi));
    }
    const float u2 = 2.f * kSqrt2OverPi * fmaf(kTanhCubic * g * g, g, g);
    const float p = logistic(u2);
    // (1 - tanh^2 u) / 2 = 2 p (1 - p)
    const float du = kSqrt2OverPi * fmaf(3.f * kTanhCubic * g, g, 1.f);
    return make_float2(g * p, fmaf(g * 2.f * p * (1.f - p), du, p));
}

}  // namespace dgb
