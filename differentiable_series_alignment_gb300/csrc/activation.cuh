// activation.cuh -- the activations of group norm and of gated linear units, and their derivatives.
#pragma once
#include "common.cuh"
#include "encoder.h"
#include "packed.cuh"

namespace sdtw {

__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// 1 / (1 + exp(-z)). EXACT, for results of 32 bits, takes expf: ex2 alone makes the rounding of its argument, up to
// |z| 2^-24, a relative error of the exponential; 16 bits do not show it.
template <bool EXACT> __device__ __forceinline__ float sigmoid(float z) {
    return reciprocal(1.f + (EXACT ? expf(-z) : ex2(-1.4426950408889634f * z)));
}

// act(z), and with SLOPE its derivative.
template <int ACT, bool EXACT, bool SLOPE> __device__ __forceinline__ float activate(float z, float& slope) {
    if constexpr (ACT == SDTW_ACT_SILU) {
        const float s = sigmoid<EXACT>(z);
        if (SLOPE) slope = fmaf(z * s, 1.f - s, s);
        return z * s;
    } else if constexpr (ACT == SDTW_ACT_GELU) {
        float c, e = 0.f;
        if constexpr (EXACT) {
            c = fmaf(0.5f, erff(z * 0.70710678118654752f), 0.5f);
            if (SLOPE) e = expf(-0.5f * z * z);
        } else {
            // Abramowitz and Stegun 7.1.26: erfc(x) = t poly(t) exp(-x^2) to 1.5e-7, whose exponential the derivative has
            // use for too
            const float t = reciprocal(fmaf(fabsf(z), 0.3275911f * 0.70710678118654752f, 1.f));
            e = ex2(-0.72134752044448170f * z * z);
            const float half = t * e * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 0.5f * 1.061405429f, 0.5f * -1.453152027f), 0.5f * 1.421413741f), 0.5f * -0.284496736f),
                                            0.5f * 0.254829592f);
            c = z < 0.f ? half : 1.f - half;
        }
        if (SLOPE) slope = fmaf(z * 0.39894228040143268f, e, c);
        return z * c;
    } else if constexpr (ACT == SDTW_ACT_RELU) {
        if (SLOPE) slope = z > 0.f ? 1.f : 0.f;
        return z < 0.f ? 0.f : z;   // NaN stays
    } else if constexpr (ACT == SDTW_ACT_SIGMOID) {
        const float s = sigmoid<EXACT>(z);
        if (SLOPE) slope = s * (1.f - s);
        return s;
    } else {
        if (SLOPE) slope = 1.f;
        return z;
    }
}

// Two values at a time: act of z, or its derivative.
template <int ACT, bool EXACT, bool SLOPE> __device__ __forceinline__ Pair activate2(Pair z) {
    float x, y, slope;
    if constexpr (ACT == SDTW_ACT_NONE) {
        return SLOPE ? pk2(1.f, 1.f) : z;
    } else if constexpr (ACT == SDTW_ACT_SILU && !EXACT) {
        upk2(mul2(z, pk2(-1.4426950408889634f, -1.4426950408889634f)), x, y);
        upk2(add2(pk2(ex2(x), ex2(y)), pk2(1.f, 1.f)), x, y);
        const Pair s = pk2(reciprocal(x), reciprocal(y)), v = mul2(z, s);
        return SLOPE ? fma2(v, sub2(pk2(1.f, 1.f), s), s) : v;
    } else {
        upk2(z, x, y);
        const float u = activate<ACT, EXACT, SLOPE>(x, slope);
        x = SLOPE ? slope : u;
        const float v = activate<ACT, EXACT, SLOPE>(y, slope);
        y = SLOPE ? slope : v;
        return pk2(x, y);
    }
}

}  // namespace sdtw
