// linear16.cu: the linear layer on 16-bit values, Y = act(X op(W) + b) + R, and the products
// and reductions of its gradient.
#include "epilogue.cuh"
#include "half16.cuh"
#include "layer16.cuh"
#include "pair_gemm16.cuh"

#include <algorithm>

namespace sg {
namespace {

// ---- K == 0: D = act(bias) + res ----------------------------------------------------------------
template <typename T>
__global__ void __launch_bounds__(256) no_product_kernel(const Gemm16 g) {
    using H = Half16<T>;
    for (long long m = blockIdx.y; m < g.M; m += gridDim.y)
        for (long long n = blockIdx.x * 256LL + threadIdx.x; n < g.N; n += gridDim.x * 256LL) {
            const float z = g.bias ? H::widen(g.bias[n]) : 0.0f;
            if (g.pre) g.pre[m * g.ldz + n] = H::narrow(z);
            float y = activate(z, g.act);
            if (g.res) y += H::widen(g.res[m * g.ldr + n]);
            g.D[m * g.ldd + n] = H::narrow(y);
        }
}

// ---- operands TMA cannot address ----------------------------------------------------------------
//
// A matrix whose base or leading dimension is not a multiple of 16 bytes is copied once into
// scratch with an aligned leading dimension, at memory speed, and the product runs on the copy.
// A thread writes 8 values from the aligned 4-byte words around them.
struct PackJob {
    const uint16_t *src;
    long long ld;
    uint16_t *dst;
    long long ldd;
    int rows, cols, gx, gy;
};

__global__ void __launch_bounds__(256) pack16_kernel(const PackJob j0, const PackJob j1) {
    const int first = j0.gx * j0.gy;
    const bool second = static_cast<int>(blockIdx.x) >= first;
    const PackJob &j = second ? j1 : j0;
    const int bid = static_cast<int>(blockIdx.x) - (second ? first : 0);
    const int bx = bid % j.gx, by = bid / j.gx;
    for (long long r = by; r < j.rows; r += j.gy)
        for (long long c = 8 * (bx * 256LL + threadIdx.x); c < j.cols; c += 2048LL * j.gx)
            *reinterpret_cast<uint4 *>(j.dst + r * j.ldd + c) =
                load8_any(j.src + r * j.ld + c, static_cast<int>(min(8LL, j.cols - c)));
}

PackJob pack_job(const uint16_t *src, long long ld, int rows, int cols, uint16_t *dst) {
    PackJob j{src, ld, dst, (cols + 7LL) / 8 * 8, rows, cols, 0, 0};
    // About 2,048 CTAs per matrix, each looping over several rows (as the fp32 repack does).
    j.gx = static_cast<int>(std::min<long long>((cols + 2047LL) / 2048, 8));
    j.gy = static_cast<int>(std::min<long long>(rows, 2048 / j.gx));
    return j;
}

// ---- dz = dy * act'(z) and its column sums --------------------------------------------------

// act'(z) * g. ReLU selects, so that an infinite gradient behind a closed gate gives zero.
__device__ __forceinline__ float activate_grad(float z, float g, int act) {
    switch (act) {
        case kActRelu: return z <= 0.0f ? 0.0f : g;
        case kActGelu:  // Phi(z) + z phi(z)
            return g * (0.5f * (1.0f + erff(z * 0.70710678118654752f)) +
                        z * 0.39894228040143268f * expf(-0.5f * z * z));
        case kActGeluTanh: {
            const float t = tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z));
            const float du = 0.79788456080286536f * (1.0f + 0.134145f * z * z);
            return g * (0.5f * (1.0f + t) + 0.5f * z * (1.0f - t * t) * du);
        }
        case kActSilu: {
            const float s = 1.0f / (1.0f + expf(-z));
            return g * s * (1.0f + z * (1.0f - s));
        }
        default: return g;
    }
}

constexpr int kSumRows = 256;  // rows of one CTA's column sums

// CTA (x, y): columns [32 x, 32 x + 32), rows [kSumRows y, ...). The CTA's sums go to
// part[y][n]; column_sum_kernel adds them over y in ascending order, so that the result does
// not depend on the order in which CTAs finish.
template <typename T>
__global__ void __launch_bounds__(256) act_grad_kernel(const ActGrad g, float *part) {
    using H = Half16<T>;
    __shared__ float sums[8][33];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const long long n = static_cast<long long>(blockIdx.x) * 32 + lane;
    const long long r0 = static_cast<long long>(blockIdx.y) * kSumRows;
    const long long r1 = min(r0 + kSumRows, static_cast<long long>(g.M));
    float sum = 0.0f;
    if (n < g.N)
        for (long long r = r0 + w; r < r1; r += 8) {
            float v = H::widen(g.dy[r * g.lddy + n]);
            if (g.act != kActNone) v = activate_grad(H::widen(g.z[r * g.ldz + n]), v, g.act);
            if (g.dz) g.dz[r * g.lddz + n] = H::narrow(v);
            sum = __fadd_rn(sum, v);  // never fused with v's last product: one result with and without dz
        }
    if (!part) return;
    sums[w][lane] = sum;
    __syncthreads();
    if (w == 0 && n < g.N) {
        for (int i = 1; i < 8; ++i) sum += sums[i][lane];
        part[static_cast<long long>(blockIdx.y) * g.N + n] = sum;
    }
}

__global__ void column_sum_kernel(const float *part, int parts, int N, float *db) {
    const long long n = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
    if (n >= N) return;
    float s = 0.0f;
    for (int i = 0; i < parts; ++i) s += part[static_cast<long long>(i) * N + n];
    db[n] = s;
}

}  // namespace

cudaError_t gemm16_launch(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    cudaError_t err = cudaSuccess;
    if (g.K == 0) {
        const dim3 grid(static_cast<unsigned>(std::min<long long>((g.N + 255LL) / 256, 64)),
                        static_cast<unsigned>(std::min(g.M, 65535)));
        if (g.dtype == kBf16)
            no_product_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(g);
        else
            no_product_kernel<__half><<<grid, 256, 0, stream>>>(g);
        err = cudaGetLastError();
        if (err != cudaSuccess) *detail = "linear layer kernel launch failed";
        return err;
    }
    Gemm16 q = g;
    const bool pack_a = !tma_rows(g.A, g.lda), pack_b = !tma_rows(g.B, g.ldb);
    if (pack_a || pack_b) {
        const int ra = g.a_mn ? g.K : g.M, ca = g.a_mn ? g.M : g.K;
        const int rb = g.b_mn ? g.K : g.N, cb = g.b_mn ? g.N : g.K;
        const size_t na = pack_a ? static_cast<size_t>(ra) * ((ca + 7LL) / 8 * 8) : 0;
        const size_t nb = pack_b ? static_cast<size_t>(rb) * ((cb + 7LL) / 8 * 8) : 0;
        void *ptr = nullptr;
        err = layer_scratch(kScratchPack, stream, (na + nb) * 2, &ptr, detail);
        if (err != cudaSuccess) return err;
        uint16_t *dst = static_cast<uint16_t *>(ptr);
        PackJob jobs[2] = {};
        int n = 0;
        if (pack_a) {
            jobs[n] = pack_job(g.A, g.lda, ra, ca, dst);
            q.A = dst;
            q.lda = jobs[n++].ldd;
        }
        if (pack_b) {
            jobs[n] = pack_job(g.B, g.ldb, rb, cb, dst + na);
            q.B = dst + na;
            q.ldb = jobs[n++].ldd;
        }
        const int blocks = jobs[0].gx * jobs[0].gy + jobs[1].gx * jobs[1].gy;
        pack16_kernel<<<blocks, 256, 0, stream>>>(jobs[0], jobs[1]);
        err = cudaGetLastError();
        if (err != cudaSuccess) {
            *detail = "repacking kernel launch failed";
            return err;
        }
    }
    return stream_gemm16_supports(q) ? stream_gemm16_launch(q, stream, detail)
                                     : pair_gemm16_launch(q, stream, detail);
}

cudaError_t act_grad_launch(const ActGrad &g, cudaStream_t stream, const char **detail) {
    const int parts = static_cast<int>((g.M + static_cast<long long>(kSumRows) - 1) / kSumRows);
    float *part = nullptr;
    cudaError_t err = cudaSuccess;
    if (g.db && g.M > 0) {
        void *p = nullptr;
        err = layer_scratch(kScratchSums, stream,
                            static_cast<size_t>(parts) * static_cast<size_t>(g.N) * 4, &p, detail);
        if (err != cudaSuccess) return err;
        part = static_cast<float *>(p);
    }
    if (g.M > 0) {
        if (parts > 65535) {
            *detail = "too many rows";
            return cudaErrorInvalidValue;
        }
        const dim3 grid(static_cast<unsigned>((g.N + 31LL) / 32), static_cast<unsigned>(parts));
        if (g.dtype == kBf16)
            act_grad_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(g, part);
        else
            act_grad_kernel<__half><<<grid, 256, 0, stream>>>(g, part);
    }
    if (g.db)
        column_sum_kernel<<<static_cast<unsigned>((g.N + 255LL) / 256), 256, 0, stream>>>(
            part, g.M > 0 ? parts : 0, g.N, g.db);
    err = cudaGetLastError();
    if (err != cudaSuccess) *detail = "gradient kernel launch failed";
    return err;
}

}  // namespace sg
