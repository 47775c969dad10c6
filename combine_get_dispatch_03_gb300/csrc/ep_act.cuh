// ep_act.cuh -- the activations of products with an epilogue, and their derivatives, in fp32.
#pragma once

#include "ep_common.cuh"

namespace ep {

// 1 / (1 + exp(-v)), to about 2^-22: log2(e) in two parts, so that the exponent's rounding comes back as a factor.  Below
// -88 it is 0 (6e-39 at -88).
__device__ __forceinline__ float sigmoid_fp32(float v) {
    constexpr float kHi = 1.44269502f, kLo = 1.92596303e-8f, kLn2 = 0.693147182f;
    const float x = fminf(fmaxf(-v, -104.0f), 88.0f);
    const float t = x * kHi;
    const float rest = fmaf(x, kHi, -t) + x * kLo;
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
    const float s = __frcp_rn(1.0f + fmaf(e, rest * kLn2, e));
    return v >= -88.0f ? s : v < -88.0f ? 0.0f : v;  // the clamps drop NaN
}

// The normal distribution up to v.  By erfc: 1 + erf loses the lower tail, where gelu's values are small but bf16 holds them.
// There erfc(x) changes by -2 x of itself with x, and what x = -v / sqrt(2) lost in its rounding comes back so (at v = -12
// 1.7e-5 of the value otherwise).
__device__ __forceinline__ float normal_cdf(float v) {
    constexpr float kHi = -0.707106769f, kLo = -1.21016175e-8f;
    const float x = v * kHi;
    const float rest = fmaf(v, kHi, -x) + v * kLo;
    const float c = 0.5f * erfcf(x);
    return x > 0.0f && x < 20.0f ? c * fmaf(-2.0f * x, rest, 1.0f) : c;
}

__device__ __forceinline__ float activate(int act, float v) {
    switch (act) {
        case EP_ACT_RELU: return v < 0.0f ? 0.0f : v;
        case EP_ACT_SILU: return v * sigmoid_fp32(v);
        case EP_ACT_GELU: return v * normal_cdf(v);
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
            const float c = normal_cdf(v);
            return make_float2(v * c, c + v * (0.398942280f * expf(-0.5f * v * v)));
        }
        default: return make_float2(v, 1.0f);
    }
}

}  // namespace ep
