// checkpoint8.cu: 16-bit matrices to 8-bit checkpoints and back (checkpoint8.cuh has the form).
#include "checkpoint8.cuh"
#include "layer16.cuh"

#include <algorithm>

namespace sg {
namespace {

// A thread has 8 consecutive columns of a row, eight threads a block of 64.
template <typename T>
__global__ void __launch_bounds__(256) save8_kernel(const Checkpoint8 c) {
    using H = Half16<T>;
    grid_dependents();
    grid_dependency();
    const long long chunks = (c.N + 63LL) / 64 * 8;  // per row, of 8 columns
    const long long total = chunks * c.M;
    const long long step = static_cast<long long>(gridDim.x) * 256;
    // Whole warps go round together: the lanes of a block exchange their maxima.
    for (long long first = blockIdx.x * 256LL; first < total; first += step) {
        const long long i = first + threadIdx.x;
        const long long row = i / chunks, chunk = i - row * chunks;
        const int col = static_cast<int>(chunk * 8);
        const int count = i < total ? static_cast<int>(max(0LL, min(8LL, c.N - chunk * 8))) : 0;
        float v[8];
        float a = 0.0f;
        bool nan = false;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (count > 0) w = load8_any(c.X + row * c.ldx + col, count);
        const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = H::widen2(words[k]);
            v[2 * k] = 2 * k < count ? f.x : 0.0f;
            v[2 * k + 1] = 2 * k + 1 < count ? f.y : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            nan |= v[k] != v[k];
            a = fmaxf(a, fabsf(v[k]));
        }
        if (nan) a = __int_as_float(0x7f800000);
#pragma unroll
        for (int s = 1; s < 8; s *= 2) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, s));
        const Coder8 coder(a);
        if (count <= 0) continue;
        int8_t *q = c.Q + row * c.ldq + col;
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < count) q[k] = static_cast<int8_t>(coder.code(v[k]));
        if ((chunk & 7) == 0) c.S[row * c.lds + chunk / 8] = coder.scale;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) restore8_kernel(const Restore8 c) {
    using H = Half16<T>;
    grid_dependents();
    grid_dependency();
    for (long long row = blockIdx.y; row < c.M; row += gridDim.y)
        for (long long col = blockIdx.x * 256LL + threadIdx.x; col < c.N; col += gridDim.x * 256LL) {
            const float s = c.S[row * c.lds + col / kCheckpointBlock];
            c.X[row * c.ldx + col] = H::narrow(decode8(static_cast<uint8_t>(c.Q[row * c.ldq + col]), s));
        }
}

}  // namespace

cudaError_t save8_launch(const Checkpoint8 &c, cudaStream_t stream, const char **detail) {
    const long long threads = (c.N + 63LL) / 64 * 8 * c.M;
    const unsigned grid = static_cast<unsigned>(std::min<long long>((threads + 255) / 256, 1 << 20));
    const cudaError_t err = launch_early(c.dtype == kBf16 ? save8_kernel<__nv_bfloat16> : save8_kernel<__half>,
                                         dim3(grid), 256, 0, stream, c);
    if (err != cudaSuccess) *detail = "checkpoint kernel launch failed";
    return err;
}

cudaError_t restore8_launch(const Restore8 &c, cudaStream_t stream, const char **detail) {
    const dim3 grid(static_cast<unsigned>(std::min<long long>((c.N + 255LL) / 256, 64)),
                    static_cast<unsigned>(std::min(c.M, 65535)));
    const cudaError_t err = launch_early(
        c.dtype == kBf16 ? restore8_kernel<__nv_bfloat16> : restore8_kernel<__half>, grid, 256, 0, stream, c);
    if (err != cudaSuccess) *detail = "restore kernel launch failed";
    return err;
}

}  // namespace sg
