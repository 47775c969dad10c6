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

// Two values at a time: a packed instruction does both.
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// exp(v) of two v in [-104, 88].
__device__ __forceinline__ float2 exp_fp32(float2 v, float2 lost) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float2 t = __fmul2_rn(v, both(kHi));
    const float2 rest = __ffma2_rn(lost, both(kHi), __ffma2_rn(v, both(kLo), __ffma2_rn(v, both(kHi), make_float2(-t.x, -t.y))));
    float2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(t.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(t.y));
    return __ffma2_rn(e, __fmul2_rn(rest, both(kLn2)), e);
}

// v, not below `low` or above `high`; NaN stays NaN.
__device__ __forceinline__ float clamp_nan(float v, float low, float high) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(low));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(high));
    return r;
}

// 1 / (1 + exp(-v)) of two, to 2^-21; below -87.3, where it passes 2^-126, 0.
__device__ __forceinline__ float2 sigmoid_fp32(float2 v) {
    const float2 c = make_float2(clamp_nan(-v.x, -104.0f, 88.0f), clamp_nan(-v.y, -104.0f, 88.0f));
    const float2 d = __fadd2_rn(exp_fp32(c, both(0.0f)), both(1.0f));
    return make_float2(reciprocal(d.x), reciprocal(d.y));
}

// The normal distribution at two v, and its density.  The smaller tail, exp(-v^2 / 2) * t * P(t) with t = 1 / (1 + 0.28 |v|),
// where P is a polynomial fitted (least maximum of the relative error, 9.1e-8 over |v| < 60) to
// 0.5 * exp(v^2 / 2) * erfc(|v| / sqrt(2)) / t; 4e-7 of the tail in fp32, at any v: 1 + erf(v) would lose the lower one, where
// gelu's values are small but bf16 holds them.  The square's rounding goes into the exponential.
__device__ __forceinline__ float2 normal_fp32(float2 v, float2* density) {
    const float2 u = make_float2(fminf(fabsf(v.x), 14.0f), fminf(fabsf(v.y), 14.0f));  // the tail is 0 from 13.2 on
    const float2 d = __ffma2_rn(u, both(0.28f), both(1.0f));
    const float2 t = make_float2(reciprocal(d.x), reciprocal(d.y));
    float2 p = both(0.0259195454f);
    p = __ffma2_rn(p, t, both(-0.0983238742f));
    p = __ffma2_rn(p, t, both(0.100072779f));
    p = __ffma2_rn(p, t, both(-0.0129762348f));
    p = __ffma2_rn(p, t, both(0.0759411454f));
    p = __ffma2_rn(p, t, both(0.0827578530f));
    p = __ffma2_rn(p, t, both(0.103213914f));
    p = __ffma2_rn(p, t, both(0.111690849f));
    p = __ffma2_rn(p, t, both(0.111704066f));
    const float2 h = __fmul2_rn(u, both(-0.5f)), q = __fmul2_rn(h, u);
    const float2 e = exp_fp32(q, __ffma2_rn(h, u, make_float2(-q.x, -q.y)));
    const float2 tail = __fmul2_rn(__fmul2_rn(e, t), p);
    *density = __fmul2_rn(e, both(0.398942280f));
    return make_float2(v.x > 0.0f ? 1.0f - tail.x : tail.x, v.y > 0.0f ? 1.0f - tail.y : tail.y);
}

// The activation of two values.
__device__ __forceinline__ float2 activate(int act, float2 v) {
    switch (act) {
        case EP_ACT_RELU: return make_float2(v.x < 0.0f ? 0.0f : v.x, v.y < 0.0f ? 0.0f : v.y);
        case EP_ACT_SILU: return __fmul2_rn(v, sigmoid_fp32(v));
        case EP_ACT_GELU: {
            float2 density;
            return __fmul2_rn(v, normal_fp32(v, &density));
        }
        default: return v;
    }
}

// And its derivative.
__device__ __forceinline__ float2 activate_with_slope(int act, float2 v, float2* slope) {
    switch (act) {
        case EP_ACT_RELU:
            *slope = make_float2(v.x > 0.0f ? 1.0f : 0.0f, v.y > 0.0f ? 1.0f : 0.0f);
            return make_float2(v.x < 0.0f ? 0.0f : v.x, v.y < 0.0f ? 0.0f : v.y);
        case EP_ACT_SILU: {
            const float2 s = sigmoid_fp32(v);
            *slope = __fmul2_rn(s, __ffma2_rn(v, __ffma2_rn(s, both(-1.0f), both(1.0f)), both(1.0f)));
            return __fmul2_rn(v, s);
        }
        case EP_ACT_GELU: {
            float2 density;
            const float2 n = normal_fp32(v, &density);
            *slope = __ffma2_rn(v, density, n);
            return __fmul2_rn(v, n);
        }
        default: *slope = both(1.0f); return v;
    }
}

}  // namespace ep
