// moe16.cuh: parts shared by the mixture-of-experts kernels.
#pragma once

#include "layer16.cuh"

namespace sg {

// The router's scores as unsigned integers of the same order: NaN above everything, -0 equal to +0.
__device__ __forceinline__ unsigned int moe_score_order(float s) {
    const unsigned int u = __float_as_uint(s == 0.0f ? 0.0f : s);
    return s != s ? 0xFFFFFFFFu : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
// The score of such an integer (NaN gives a NaN).
__device__ __forceinline__ float moe_order_score(unsigned int u) {
    return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}
// With the index below it, so that equal scores go to the lowest expert.
__device__ __forceinline__ unsigned long long moe_score_key(float s, int e) {
    return (static_cast<unsigned long long>(moe_score_order(s)) << 32) | (0xFFFFFFFFu - static_cast<unsigned>(e));
}

// The fused kernel: needs operands TMA can address.
bool moe_stream_supports(const Moe16 &m);
cudaError_t moe_stream_launch(const Moe16 &m, cudaStream_t stream, const char **detail);

}  // namespace sg
