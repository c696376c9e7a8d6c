// checkpoint8.cuh: the 8-bit form in which activations are kept for the backward pass.
//
// A row's blocks of 64 consecutive columns share a scale: with a the block's largest magnitude,
// s = a / 127 (fp32, rounded once) and q = 127 x / a rounded to the nearest integer, ties to even;
// q s, rounded to the 16-bit type, is the restored value. A block of zeros has s = 0. One that holds an
// infinity or a NaN has s = NaN and q = 0, so that it restores to NaN. 64 columns: what one epilogue warp
// of the pair product has of a row, and 1.06 bytes a value.
#pragma once

#include "half16.cuh"

namespace sg {

constexpr int kCheckpointBlock = 64;

// The largest magnitude among 16-bit values, as bits without the sign: they order as integers, with
// infinity and then NaN above every finite value. `acc` holds two candidates, `w` two values.
template <typename T>
__device__ __forceinline__ uint32_t magnitude2(uint32_t acc, uint32_t w) {
    w &= 0x7FFF7FFFu;
    if constexpr (Half16<T>::kind == kBf16) {
        const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&acc),
                                             *reinterpret_cast<const __nv_bfloat162 *>(&w));
        return *reinterpret_cast<const uint32_t *>(&m);
    } else {
        const __half2 m = __hmax2_nan(*reinterpret_cast<const __half2 *>(&acc), *reinterpret_cast<const __half2 *>(&w));
        return *reinterpret_cast<const uint32_t *>(&m);
    }
}
__device__ __forceinline__ uint32_t magnitude(uint32_t acc) { return max(acc & 0xFFFFu, acc >> 16); }

template <typename T>
__device__ __forceinline__ bool is_finite(uint32_t magnitude_bits) {
    return magnitude_bits < (Half16<T>::kind == kBf16 ? 0x7F80u : 0x7C00u);
}
// What is stored for a block whose largest magnitude has the bits `top`.
template <typename T>
__device__ __forceinline__ float scale8(uint32_t top) {
    return is_finite<T>(top) ? __fdiv_rn(Half16<T>::widen(static_cast<uint16_t>(top)), 127.0f)
                             : __int_as_float(0x7fc00000);
}

// The codes of such a block, from its inverse 127 / a in two fp32 parts. x (hi + lo) is then within 2^-36 of the
// quotient, and its one rounding to fp32 moves no value onto or over a tie: with x in [a 2^-s-1, a 2^-s] the
// quotient is (k + 1/2) exactly, which fp32 holds, or differs from it by at least 2^-12-s (both have at most 11
// significant bits), 16 times its fp32 spacing. (A product with a rounded inverse is off at ties, which are
// not rare: every 300th normal bfloat16 value is one.)
template <typename T>
struct Coder8 {
    float hi, lo, lift;
    bool finite;
    __device__ __forceinline__ explicit Coder8(uint32_t top) {
        float a = Half16<T>::widen(static_cast<uint16_t>(top));
        finite = is_finite<T>(top);
        // 127 / a could overflow, or leave the range of the approximate division
        lift = !finite || a > 1e30f ? 5.42101086e-20f : a < 1e-30f ? 18446744073709551616.0f : 1.0f;  // 2^-64, 2^64
        a *= lift;
        hi = __fdividef(127.0f, a);
        lo = __fdividef(fmaf(-hi, a, 127.0f), a);
        if (!(a > 0.0f)) hi = lo = 0.0f;
    }
    // Eight codes, two's complement, lowest byte first.
    __device__ __forceinline__ uint2 eight(const uint32_t (&w)[4]) const {
        if (lift == 1.0f) return round8<false>(w);
        return finite ? round8<true>(w) : make_uint2(0, 0);
    }

private:
    template <bool LIFT>
    __device__ __forceinline__ uint2 round8(const uint32_t (&w)[4]) const {
        uint32_t bits[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float2 f = Half16<T>::widen2(w[i]);
            if (LIFT) f = __fmul2_rn(f, make_float2(lift, lift));
            const float2 q = __ffma2_rn(f, make_float2(hi, hi), __fmul2_rn(f, make_float2(lo, lo)));
            // 1.5 2^23: the sum's low bits are the nearest integer, ties to even
            const float2 m = __fadd2_rn(q, make_float2(12582912.0f, 12582912.0f));
            bits[2 * i] = __float_as_uint(m.x);
            bits[2 * i + 1] = __float_as_uint(m.y);
        }
        auto four = [](const uint32_t *b) {
            return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
        };
        return make_uint2(four(bits), four(bits + 4));
    }
};

// The restored values of four codes, in 16 bits: the bytes, made unsigned, become the low bits of 2^23 +
// byte, from which the difference is exact.
template <typename T>
__device__ __forceinline__ uint2 restore4(uint32_t word, float2 s01, float2 s23) {
    const uint32_t b = word ^ 0x80808080u;
    auto at = [&](int k) { return __uint_as_float(__byte_perm(b, 0x4B000000u, 0x7540 + k)); };
    const float2 bias = make_float2(-8388736.0f, -8388736.0f);  // 2^23 + 128
    const float2 lo = __fmul2_rn(__fadd2_rn(make_float2(at(0), at(1)), bias), s01);
    const float2 hi = __fmul2_rn(__fadd2_rn(make_float2(at(2), at(3)), bias), s23);
    return make_uint2(Half16<T>::narrow2(lo.x, lo.y), Half16<T>::narrow2(hi.x, hi.y));
}

}  // namespace sg
