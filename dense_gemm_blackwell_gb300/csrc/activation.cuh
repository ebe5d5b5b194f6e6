// activation.cuh -- the activations of a gated feed-forward block and their
// slopes, in fp32.
#pragma once

#include "elem.cuh"
#include "feedforward.h"

namespace dgb {

// 1 / (1 + e^-x): 0 for a very negative x (e^-x infinite).
__device__ __forceinline__ float logistic(float x) { return __fdividef(1.f, 1.f + exp2_fast(-1.4426950408889634f * x)); }

// Q(|g|) = e^(-g^2/2) R(|g|), the normal distribution's upper tail, with e^(-g^2/2) given.  R(z) = erfc(z / sqrt 2) e^(z^2/2) / 2
// is smooth in t = 1 / (1 + 0.3 z): t times a polynomial of degree 7, fitted to the least relative error over 0 <= z <= 14
// (where Q leaves fp32's range), 1.5e-7; 5e-7 as evaluated in fp32.  CUDA's erfcf in the pipeline's epilogue cost 7.6 of 19.9 us
// at 777 x 1001 x 2 * 1544.
__device__ __forceinline__ float normal_tail(float g, float e) {
    const float t = __fdividef(1.f, fmaf(0.3f, fabsf(g), 1.f));
    float p = fmaf(3.567481413e-2f, t, -1.572032422e-1f);
    p = fmaf(p, t, 2.063537687e-1f);
    p = fmaf(p, t, -5.368387327e-2f);
    p = fmaf(p, t, 1.285617352e-1f);
    p = fmaf(p, t, 9.991346300e-2f);
    p = fmaf(p, t, 1.207539588e-1f);
    p = fmaf(p, t, 1.196293011e-1f);
    return e * t * p;
}

constexpr float kSqrt2OverPi = 0.7978845608028654f, kTanhCubic = 0.044715f;

// silu: g / (1 + e^-g).  gelu: g Phi(g), from the tail that g lies in, which keeps its accuracy for negative g, where 1 + erf
// cancels.  gelu_tanh: g (1 + tanh u) / 2 = g / (1 + e^-2u), u = sqrt(2/pi) (g + 0.044715 g^3).
__device__ __forceinline__ float activate(int act, float g) {
    if (act == GATED_SILU) return g * logistic(g);
    if (act == GATED_GELU) {
        const float q = normal_tail(g, exp2_fast(-0.7213475204444817f * g * g));
        return g * (g < 0.f ? q : 1.f - q);
    }
    return g * logistic(2.f * kSqrt2OverPi * fmaf(kTanhCubic * g * g, g, g));
}

// The activation and its derivative.
__device__ __forceinline__ float2 activate_with_slope(int act, float g) {
    if (act == GATED_SILU) {
        const float p = logistic(g);
        return make_float2(g * p, p * fmaf(g, 1.f - p, 1.f));
    }
    if (act == GATED_GELU) {
        const float e = exp2_fast(-0.7213475204444817f * g * g), q = normal_tail(g, e);
        const float phi = g < 0.f ? q : 1.f - q;
        return make_float2(g * phi, fmaf(g * 0.3989422804014327f, e, phi));      // + g e^(-g^2/2) / sqrt(2 pi)
    }
    const float u2 = 2.f * kSqrt2OverPi * fmaf(kTanhCubic * g * g, g, g);
    const float p = logistic(u2);
    // (1 - tanh^2 u) / 2 = 2 p (1 - p): 0 long before |g| = 64, past which du might overflow
    const float near = fminf(fmaxf(g, -64.f), 64.f), du = kSqrt2OverPi * fmaf(3.f * kTanhCubic * near, near, 1.f);
    return make_float2(g * p, fmaf(near * 2.f * p * (1.f - p), du, p));
}

}  // namespace dgb
