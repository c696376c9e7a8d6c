// half16.cuh: 16-bit storage types (bfloat16, IEEE half) of the layer operators. Values are
// widened exactly to fp32 when read and rounded once, to nearest even, when written.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace sg {

enum Dtype16 : int { kBf16 = 0, kF16 = 1 };

template <typename T>
struct Half16;

template <>
struct Half16<__nv_bfloat16> {
    static constexpr int kind = kBf16;
    __device__ static __forceinline__ float widen(uint16_t v) {
        return __uint_as_float(static_cast<uint32_t>(v) << 16);
    }
    __device__ static __forceinline__ uint16_t narrow(float v) {
        return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    }
    __device__ static __forceinline__ float2 widen2(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    // lo in the low half
    __device__ static __forceinline__ uint32_t narrow2(float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

template <>
struct Half16<__half> {
    static constexpr int kind = kF16;
    __device__ static __forceinline__ float widen(uint16_t v) {
        return __half2float(__ushort_as_half(v));
    }
    __device__ static __forceinline__ uint16_t narrow(float v) {
        return __half_as_ushort(__float2half_rn(v));
    }
    __device__ static __forceinline__ float2 widen2(uint32_t v) {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    __device__ static __forceinline__ uint32_t narrow2(float lo, float hi) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// 8 values of a row at any 2-byte aligned address, of which the first `count` (up to 8) belong to
// the row: first the aligned 4-byte words that hold one of them (load8_words, so that several
// loads can be under way), then the values from the words (align8; past `count` arbitrary).
__device__ __forceinline__ void load8_words(uint32_t (&v)[5], const uint16_t *src, int count) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(src);
    const int shift = static_cast<int>(a & 2u) >> 1;  // the first word's low half precedes the row
    const uint32_t *w = reinterpret_cast<const uint32_t *>(a & ~static_cast<uintptr_t>(3));
#pragma unroll
    for (int i = 0; i < 5; ++i)
        if (2 * i - shift < count) v[i] = __ldg(w + i);
}
__device__ __forceinline__ uint4 align8(const uint32_t (&v)[5], const uint16_t *src) {
    if (reinterpret_cast<uintptr_t>(src) & 2u)
        return make_uint4(__funnelshift_r(v[0], v[1], 16), __funnelshift_r(v[1], v[2], 16),
                          __funnelshift_r(v[2], v[3], 16), __funnelshift_r(v[3], v[4], 16));
    return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint4 load8_any(const uint16_t *src, int count) {
    if ((reinterpret_cast<uintptr_t>(src) & 15u) == 0 && count == 8)
        return __ldg(reinterpret_cast<const uint4 *>(src));
    uint32_t v[5] = {};
    load8_words(v, src, count);
    return align8(v, src);
}

}  // namespace sg
