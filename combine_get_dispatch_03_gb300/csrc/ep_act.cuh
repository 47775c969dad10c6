// ep_act.cuh -- the activations of products with an epilogue, and their derivatives, in fp32.
#pragma once

#include "ep_common.cuh"

namespace ep {

// exp(v) for v in [-104, 88], to 2^-22: log2(e) in two parts, so that the exponent's rounding comes back as a factor; `lost`
// is what v itself lacks.  Below 2^-126 it is 0.
__device__ __forceinline__ float exp_fp32(float v, float lost = 0.0f) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float t = v * kHi;
    const float rest = fmaf(v, kHi, -t) + fmaf(v, kLo, lost * kHi);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    return fmaf(e, rest * kLn2, e);
}

__device__ __forceinline__ float reciprocal(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// 1 / (1 + exp(-v)), to 2^-21; below -87.3, where it passes 2^-126, 0.
__device__ __forceinline__ float sigmoid_fp32(float v) {
    const float s = reciprocal(1.0f + exp_fp32(fminf(fmaxf(-v, -104.0f), 88.0f)));
    return v >= -88.0f ? s : v < -88.0f ? 0.0f : v;  // the clamps drop NaN
}

// The normal distribution and its density at v.  The smaller tail, exp(-v^2 / 2) * t * P(t) with t = 1 / (1 + 0.28 |v|), where
// P is a polynomial fitted (least maximum of the relative error, 9.1e-8 over |v| < 60) to 0.5 * exp(v^2 / 2) * erfc(|v| / sqrt(2)) / t;
// 4e-7 of the tail in fp32, at any v: 1 + erf(v) would lose the lower one, where gelu's values are small but bf16 holds
// them.  The square's rounding goes into the exponential.
__device__ __forceinline__ float2 normal_fp32(float v) {
    const float u = fminf(fabsf(v), 14.0f);  // the tail is 0 from 13.2 on
    const float t = reciprocal(fmaf(0.28f, u, 1.0f));
    float p = 0.0259195454f;
    p = fmaf(p, t, -0.0983238742f);
    p = fmaf(p, t, 0.100072779f);
    p = fmaf(p, t, -0.0129762348f);
    p = fmaf(p, t, 0.0759411454f);
    p = fmaf(p, t, 0.0827578530f);
    p = fmaf(p, t, 0.103213914f);
    p = fmaf(p, t, 0.111690849f);
    p = fmaf(p, t, 0.111704066f);
    const float h = 0.5f * u, q = h * u;
    const float e = exp_fp32(-q, -fmaf(h, u, -q));
    const float tail = e * t * p;
    return make_float2(v > 0.0f ? 1.0f - tail : tail, 0.398942280f * e);
}

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case EP_ACT_RELU: return v < 0.0f ? 0.0f : v;
        case EP_ACT_SILU: return v * sigmoid_fp32(v);
        case EP_ACT_GELU: return v * normal_fp32(v).x;
        default: return v;
    }
}

// activate(v) and its derivative.
__device__ __forceinline__ float2 activate_with_slope(int act, float v) {
    switch (act) {
        case EP_ACT_RELU: return v > 0.0f ? make_float2(v, 1.0f) : make_float2(v < 0.0f ? 0.0f : v, 0.0f);
        case EP_ACT_SILU: {
            const float s = sigmoid_fp32(v);
            return make_float2(v * s, s * (1.0f + v * (1.0f - s)));
        }
        case EP_ACT_GELU: {
            const float2 n = normal_fp32(v);
            return make_float2(v * n.x, fmaf(v, n.y, n.x));
        }
        default: return make_float2(v, 1.0f);
    }
}

}  // namespace ep
