// linear16.cu: the linear layer on 16-bit values, Y = act(X op(W) + b) + R, and the products
// and reductions of its gradient.
#include "epilogue.cuh"
#include "half16.cuh"
#include "layer16.cuh"

#include <algorithm>

namespace sg {
namespace {

// ---- D = act(A . B + bias) + res ------------------------------------------------------------
//
// A 64 x 64 tile per CTA of 256 threads, 4 x 4 outputs per thread, fp32 FMAs over 16-wide
// k-tiles in shared memory. Any size, stride and alignment: every load and store is one value.
constexpr int kTile = 64, kTileK = 16;

template <typename T>
__global__ void __launch_bounds__(256) gemm16_simple_kernel(const Gemm16 g) {
    using H = Half16<T>;
    __shared__ float As[kTileK][kTile + 1], Bs[kTileK][kTile + 1];
    const int m0 = blockIdx.y * kTile;
    const long long n0 = static_cast<long long>(blockIdx.x) * kTile;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    const long long arow = g.a_mn ? 1 : g.lda, ak = g.a_mn ? g.lda : 1;
    const long long bcol = g.b_mn ? 1 : g.ldb, bk = g.b_mn ? g.ldb : 1;
    for (long long mb = m0; mb < g.M; mb += static_cast<long long>(gridDim.y) * kTile) {
        float acc[4][4] = {};
        for (long long k0 = 0; k0 < g.K; k0 += kTileK) {
            for (int i = threadIdx.x; i < kTile * kTileK; i += 256) {
                const int ar = g.a_mn ? i % kTile : i / kTileK, akk = g.a_mn ? i / kTile : i % kTileK;
                const long long m = mb + ar, ka = k0 + akk;
                As[akk][ar] = m < g.M && ka < g.K ? H::widen(g.A[m * arow + ka * ak]) : 0.0f;
                const int bc = g.b_mn ? i % kTile : i / kTileK, bkk = g.b_mn ? i / kTile : i % kTileK;
                const long long n = n0 + bc, kb = k0 + bkk;
                Bs[bkk][bc] = n < g.N && kb < g.K ? H::widen(g.B[n * bcol + kb * bk]) : 0.0f;
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < kTileK; ++k) {
                float a[4], b[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) a[i] = As[k][ty + 16 * i];
#pragma unroll
                for (int j = 0; j < 4; ++j) b[j] = Bs[k][tx + 16 * j];
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
            }
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const long long m = mb + ty + 16 * i;
            if (m >= g.M) continue;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const long long n = n0 + tx + 16 * j;
                if (n >= g.N) continue;
                float z = acc[i][j];
                if (g.bias) z += H::widen(g.bias[n]);
                if (g.pre) g.pre[m * g.ldz + n] = H::narrow(z);
                float y = activate(z, g.act);
                if (g.res) y += H::widen(g.res[m * g.ldr + n]);
                g.D[m * g.ldd + n] = H::narrow(y);
            }
        }
    }
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
    const long long gx = (g.N + static_cast<long long>(kTile) - 1) / kTile;
    const long long gy = std::min<long long>((g.M + static_cast<long long>(kTile) - 1) / kTile, 65535);
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy));
    if (g.dtype == kBf16)
        gemm16_simple_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(g);
    else
        gemm16_simple_kernel<__half><<<grid, 256, 0, stream>>>(g);
    const cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) *detail = "linear layer kernel launch failed";
    return err;
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
