// activation16.cuh: the activations and their derivatives for 16-bit results, in 10 to 20 fp32
// instructions each (an SM issues 128 a clock, and a layer's epilogue or gradient pass has only a
// few hundred clocks per thousand values before memory is faster than arithmetic).
//
// An activation's error is relative to its value, tails included, so that rounding the result to 16
// bits decides it: below 4e-5 |act(z)| for |z| <= 12, of which the arguments of the exponentials have
// most (half an ulp of f16 is 2.4e-4 to 4.9e-4). Values below 2^-126 become 0.
//
// The normal distribution's tail is its density times the Mills ratio, Phi(-z) = phi(z) M(z), and
// M(z) = t P(t) with t = 1 / (1 + c z), P a minimax fit over 0 <= z <= 13.5, made for this file by
// iterated reweighted least squares. (A form with a bound on Phi's absolute error is off by 1% of
// gelu(z) at z = -8.) For values, which are rounded to 16 bits, degree 5: within 5.9e-6 M. For slopes, whose
// sums leave in fp32, degree 6: within min(1e-5 M, 1.5e-8 / phi), which keeps their digits near 0 too
// (the bias' gradient over 16384 rows is 1.6e-7 off, as in plain fp32; with degree 5 1.7e-6). Degree 6
// for values costs a large product's epilogue 0.8%. The exponential is also the density that the
// derivative needs. tanh-GELU is z * sigmoid(2u). ex2.approx and rcp.approx are the hardware's own
// 2^x and 1/x (relative errors of 2^-22 and 1 ulp).
#pragma once

#include <type_traits>

#include "epilogue.cuh"

namespace sg {

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Phi(z), with exp(-z^2 / 2) in `e`.
template <bool SLOPE>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    constexpr float kDensity = 0.39894228040143268f;  // 1 / sqrt(2 pi)
    e = exp2_approx(z * z * -0.72134752044448170f);   // log2(e) / 2
    const float t = rcp_approx(fmaf(SLOPE ? 0.34f : 0.3125f, fabsf(z), 1.0f));
    float q;
    if (SLOPE) {
        q = fmaf(0.11014157f * kDensity, t, -0.49310258f * kDensity);
        q = fmaf(q, t, 0.64536417f * kDensity);
        q = fmaf(q, t, -0.062214788f * kDensity);
        q = fmaf(q, t, 0.38539791f * kDensity);
        q = fmaf(q, t, 0.32692045f * kDensity);
        q = fmaf(q, t, 0.34080744f * kDensity);
    } else {
        q = fmaf(-0.18044753f * kDensity, t, 0.42412591f * kDensity);
        q = fmaf(q, t, 0.064630046f * kDensity);
        q = fmaf(q, t, 0.32567805f * kDensity);
        q = fmaf(q, t, 0.30650491f * kDensity);
        q = fmaf(q, t, 0.31281543f * kDensity);
    }
    q *= t * e;  // the upper tail
    return z < 0.0f ? q : 1.0f - q;
}

__device__ __forceinline__ float sigmoid16(float z) {
    return rcp_approx(1.0f + exp2_approx(z * -1.4426950408889634f));
}

template <int ACT>
__device__ __forceinline__ float activate16(float z) {
    if (ACT == kActRelu) return activate(z, kActRelu);
    if (ACT == kActGelu) {
        float e;
        return z * normal_cdf<false>(z, e);
    }
    if (ACT == kActGeluTanh)
        return z * sigmoid16(1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
    if (ACT == kActSilu) return z * sigmoid16(z);
    return z;
}

// g * act'(z). ReLU selects, so that an infinite gradient behind a closed gate gives zero.
template <int ACT>
__device__ __forceinline__ float activate16_grad(float z, float g) {
    if (ACT == kActRelu) return z <= 0.0f ? 0.0f : g;
    if (ACT == kActGelu) {  // Phi(z) + z phi(z)
        float e;
        const float c = normal_cdf<true>(z, e);
        return g * fmaf(z * 0.39894228040143268f, e, c);
    }
    if (ACT == kActGeluTanh) {  // s + z s (1 - s) (2u)', 2u = 1.5957... (z + 0.044715 z^3)
        const float z2 = z * z;
        const float s = sigmoid16(1.5957691216057308f * fmaf(0.044715f * z2, z, z));
        const float w = s * (1.0f - s);
        const float d = w == 0.0f ? 0.0f : z * w * 1.5957691216057308f * fmaf(0.134145f, z2, 1.0f);
        return g * (s + d);
    }
    if (ACT == kActSilu) {
        const float s = sigmoid16(z);
        return g * s * fmaf(z, 1.0f - s, 1.0f);
    }
    return g;
}

// Calls body with the activation as a compile-time constant.
template <typename Body>
__device__ __forceinline__ void with_activation(int act, Body body) {
    switch (act) {
        case kActRelu: body(std::integral_constant<int, kActRelu>()); break;
        case kActGelu: body(std::integral_constant<int, kActGelu>()); break;
        case kActGeluTanh: body(std::integral_constant<int, kActGeluTanh>()); break;
        case kActSilu: body(std::integral_constant<int, kActSilu>()); break;
        default: body(std::integral_constant<int, kActNone>()); break;
    }
}

}  // namespace sg
