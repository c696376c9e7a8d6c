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

// The codes of a block whose largest magnitude is `a` (of the type T's values).
struct Coder8 {
    float scale;  // what is stored
    float top;    // a, or what keeps the codes of a block without a magnitude at 0
    float c;      // keeps 127 x finite
    bool finite;
    __device__ __forceinline__ explicit Coder8(float a) {
        finite = a < __int_as_float(0x7f800000);  // false for NaN
        scale = finite ? __fdiv_rn(a, 127.0f) : __int_as_float(0x7fc00000);
        c = a > 1e30f ? 0.0009765625f : 1.0f;
        top = finite && a > 0.0f ? a * c : 1.0f;
    }
    // The code's two's complement in the low 8 bits. 127 x has at most 18 significant bits, so it is exact,
    // and the quotient's rounding moves no value onto or over a tie: 127 x / a is (k + 1/2) exactly or
    // differs from it by at least 2^-21, which exceeds its fp32 rounding error where |q| < 128 asks for it.
    __device__ __forceinline__ uint32_t code(float x) const {
        const float q = finite ? __fdiv_rn(x * c * 127.0f, top) : 0.0f;
        return __float_as_uint(q + 12582912.0f) & 0xFFu;  // 1.5 2^23: the integer in the low bits
    }
};

__device__ __forceinline__ float decode8(uint32_t byte, float scale) {
    return static_cast<float>(static_cast<int8_t>(byte)) * scale;
}

}  // namespace sg
