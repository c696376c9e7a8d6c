// activation16.cuh: the activations and their derivatives for 16-bit results, in 10 to 20 fp32
// instructions each (an SM issues 128 a clock, and a layer's epilogue or gradient pass has only a
// few hundred clocks per thousand values before memory is faster than arithmetic).
//
// The normal distribution function comes from Hastings' approximation (Abramowitz & Stegun 1964,
// 7.1.26): erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2) with t = 1 / (1 + p x) for x >= 0, off by at
// most 1.5e-7; its exponential is also the density that the derivative needs. tanh-GELU is
// z * sigmoid(2u). The errors are of the order of an fp32 rounding of (1 + |z|), a thousandth of
// the rounding of the 16-bit result. __expf and __fdividef are CUDA's own.
#pragma once

#include <type_traits>

#include "epilogue.cuh"

namespace sg {

// Phi(z), with exp(-z^2 / 2) in `e`.
__device__ __forceinline__ float normal_cdf(float z, float &e) {
    const float x = fabsf(z) * 0.70710678118654752f;
    e = __expf(-x * x);
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    q = 0.5f * q * t * e;  // the upper tail
    return z < 0.0f ? q : 1.0f - q;
}

__device__ __forceinline__ float sigmoid16(float z) {
    return __fdividef(1.0f, 1.0f + __expf(-z));
}

template <int ACT>
__device__ __forceinline__ float activate16(float z) {
    if (ACT == kActRelu) return activate(z, kActRelu);
    if (ACT == kActGelu) {
        float e;
        return z * normal_cdf(z, e);
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
        const float c = normal_cdf(z, e);
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
