// linear16.cu: the linear layer on 16-bit values, Y = act(X op(W) + b) + R, and the products
// and reductions of its gradient.
#include "activation16.cuh"
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
    grid_dependents();
    grid_dependency();
    for (long long m = blockIdx.y; m < g.M; m += gridDim.y)
        for (long long n = blockIdx.x * 256LL + threadIdx.x; n < g.N; n += gridDim.x * 256LL) {
            const float z = g.bias ? H::widen(g.bias[n]) : 0.0f;
            if (g.pre) g.pre[m * g.ldz + n] = H::narrow(z);
            float y = z;
            with_activation(g.act, [&](auto act) { y = activate16<decltype(act)::value>(z); });
            if (g.res) y += H::widen(g.res[m * g.ldr + n]);
            g.D[m * g.ldd + n] = H::narrow(y);
        }
}

// ---- operands TMA cannot address ----------------------------------------------------------------
//
// A matrix whose base or leading dimension is not a multiple of 16 bytes is copied once into
// scratch with an aligned leading dimension, at memory speed, and the product runs on the copy.
// A thread writes 8 values from the aligned 4-byte words around them (X and W of 4095 x 3001 x 1537:
// 8.8 to 10.4 us for 44 MB read and written).
struct PackJob {
    const uint16_t *src;
    long long ld;
    uint16_t *dst;
    long long ldd;
    int rows, cols, gx, gy;
};

__global__ void __launch_bounds__(256) pack16_kernel(const PackJob j0, const PackJob j1) {
    grid_dependents();
    grid_dependency();
    const int first = j0.gx * j0.gy;
    const bool second = static_cast<int>(blockIdx.x) >= first;
    const PackJob &j = second ? j1 : j0;
    const int bid = static_cast<int>(blockIdx.x) - (second ? first : 0);
    const int bx = bid % j.gx, by = bid / j.gx;
    // Two rows at a time, so that twice the loads are under way.
    for (long long c = 8 * (bx * 256LL + threadIdx.x); c < j.cols; c += 2048LL * j.gx) {
        const int count = static_cast<int>(min(8LL, j.cols - c));
        for (long long r = by; r < j.rows; r += 2LL * j.gy) {
            const bool two = r + j.gy < j.rows;
            const uint16_t *s0 = j.src + r * j.ld + c, *s1 = s0 + j.gy * j.ld;
            uint32_t v0[5] = {}, v1[5] = {};
            load8_words(v0, s0, count);
            if (two) load8_words(v1, s1, count);
            uint16_t *d = j.dst + r * j.ldd + c;
            *reinterpret_cast<uint4 *>(d) = align8(v0, s0);
            if (two) *reinterpret_cast<uint4 *>(d + j.gy * j.ldd) = align8(v1, s1);
        }
    }
}

PackJob pack_job(const uint16_t *src, long long ld, int rows, int cols) {
    PackJob j{src, ld, nullptr, (cols + 7LL) / 8 * 8, rows, cols, 0, 0};
    // About 2,048 CTAs per matrix, each looping over several rows (as the fp32 repack does).
    j.gx = static_cast<int>(std::min<long long>((cols + 2047LL) / 2048, 8));
    j.gy = static_cast<int>(std::min<long long>(rows, 2048 / j.gx));
    return j;
}

// ---- dz = dy * act'(z) and its column sums --------------------------------------------------
//
// Bound by memory (two matrices read, one written; db alone, so that none is written: 16384 x 14336
// bf16 with GELU 202 us, 4.7 TB/s; 4095 x 3001 f16 in unaligned rows 20.3 us, 2.4 TB/s). A CTA
// covers 256 columns and `rows` rows: a thread 8 columns (16 bytes) of every eighth row, four rows' loads in flight at once. Its 8 fp32
// sums are added over the CTA's 8 threads of a column in a fixed order into part[row block][n], and
// the CTA that completes a column block's last part (a count in memory; nothing waits) adds the
// parts, four runs of them at once and then the runs' sums, in an order of their own, so that db
// does not depend on timing.
constexpr int kGradCols = 256;

template <bool VEC, int W>
__device__ __forceinline__ void load8_row(uint32_t (&v)[W], const uint16_t *src, int count) {
    if constexpr (VEC) {
        const uint4 q = __ldg(reinterpret_cast<const uint4 *>(src));
        v[0] = q.x;
        v[1] = q.y;
        v[2] = q.z;
        v[3] = q.w;
    } else {
        load8_words(v, src, count);
    }
}
template <bool VEC, int W>
__device__ __forceinline__ void align8_row(uint32_t (&out)[4], const uint32_t (&v)[W], const uint16_t *src) {
    if constexpr (VEC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) out[i] = v[i];
    } else {
        const uint4 q = align8(v, src);
        out[0] = q.x;
        out[1] = q.y;
        out[2] = q.z;
        out[3] = q.w;
    }
}

template <typename T, int ACT, bool VEC>
__device__ __forceinline__ void act_grad_rows(const ActGrad &g, long long r0, long long r1, int c,
                                              int count, float (&sum)[8]) {
    using H = Half16<T>;
    constexpr int UNROLL = VEC ? 4 : 2;
    for (long long r = r0; r < r1; r += 8 * UNROLL) {
        constexpr int W = VEC ? 4 : 5;
        uint32_t dy[UNROLL][W], z[UNROLL][W];
#pragma unroll
        for (int i = 0; i < UNROLL; ++i)
            if (r + 8 * i < r1) {
                load8_row<VEC>(dy[i], g.dy + (r + 8 * i) * g.lddy + c, count);
                if (ACT != kActNone) load8_row<VEC>(z[i], g.z + (r + 8 * i) * g.ldz + c, count);
            }
#pragma unroll
        for (int i = 0; i < UNROLL; ++i) {
            if (r + 8 * i >= r1) break;
            uint32_t d4[4], z4[4] = {};
            align8_row<VEC>(d4, dy[i], g.dy + (r + 8 * i) * g.lddy + c);
            if (ACT != kActNone) align8_row<VEC>(z4, z[i], g.z + (r + 8 * i) * g.ldz + c);
            uint32_t out[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float2 v = H::widen2(d4[q]);
                if (ACT != kActNone) {
                    const float2 zv = H::widen2(z4[q]);
                    v.x = activate16_grad<ACT>(zv.x, v.x);
                    v.y = activate16_grad<ACT>(zv.y, v.y);
                }
                // Never fused with the products before them: the same sums with and without dz.
                sum[2 * q] = __fadd_rn(sum[2 * q], v.x);
                sum[2 * q + 1] = __fadd_rn(sum[2 * q + 1], v.y);
                out[q] = H::narrow2(v.x, v.y);
            }
            // dz's rows are padded to 16 bytes: the values past N land in the padding.
            if (g.dz)
                *reinterpret_cast<uint4 *>(g.dz + (r + 8 * i) * g.lddz + c) =
                    make_uint4(out[0], out[1], out[2], out[3]);
        }
    }
}

// VEC: dy and z allow 16-byte loads (and N is a multiple of 8).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 3) act_grad_kernel(const ActGrad g, int rows, float *part,
                                                       unsigned int *counters) {
    __shared__ __align__(16) float sums[8][kGradCols];
    __shared__ unsigned int arrived;
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int c = blockIdx.x * kGradCols + lane * 8;
    const int count = min(8, g.N - c);
    const long long r0 = static_cast<long long>(blockIdx.y) * rows;
    const long long r1 = min(r0 + rows, static_cast<long long>(g.M));
    float sum[8] = {};
    if (count > 0)
        with_activation(g.act, [&](auto act) {
            act_grad_rows<T, decltype(act)::value, VEC>(g, r0 + w, r1, c, count, sum);
        });
    if (!g.db) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[w][lane * 8 + i] = sum[i];
    __syncthreads();
    const int n = blockIdx.x * kGradCols + threadIdx.x;
    float s = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 8; ++i) s += sums[i][threadIdx.x];
    const int parts = gridDim.y;
    if (parts == 1) {
        if (n < g.N) g.db[n] = s;
        return;
    }
    const long long ldp = static_cast<long long>(gridDim.x) * kGradCols;
    __stcg(part + blockIdx.y * ldp + n, s);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        arrived = atomicAdd(&counters[blockIdx.x], 1u);
        if (arrived == static_cast<unsigned>(parts - 1)) counters[blockIdx.x] = 0;
    }
    __syncthreads();
    if (arrived != static_cast<unsigned>(parts - 1)) return;
    __threadfence();
    // Thread (run, quad): columns 4 quad .. + 3 of every fourth part from `run` on.
    const int run = threadIdx.x >> 6, quad = threadIdx.x & 63;
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 16
    for (int i = run; i < parts; i += 4) {
        const float4 q = __ldcg(reinterpret_cast<const float4 *>(part + i * ldp + blockIdx.x * kGradCols) + quad);
        a.x += q.x;
        a.y += q.y;
        a.z += q.z;
        a.w += q.w;
    }
    *reinterpret_cast<float4 *>(&sums[run][4 * quad]) = a;
    __syncthreads();
    if (n < g.N)
        g.db[n] = (sums[0][threadIdx.x] + sums[1][threadIdx.x]) + (sums[2][threadIdx.x] + sums[3][threadIdx.x]);
}

__global__ void zero_kernel(float *p, int n) {
    grid_dependents();
    grid_dependency();
    const long long i = blockIdx.x * 256LL + threadIdx.x;
    if (i < n) p[i] = 0.0f;
}

}  // namespace

cudaError_t gemm16_launch(const Gemm16 *list, int n, cudaStream_t stream, const char **detail) {
    cudaError_t err = cudaSuccess;
    Gemm16 q[kMaxProducts];
    int products = 0;
    for (int i = 0; i < n; ++i) {
        const Gemm16 &g = list[i];
        if (g.K > 0) {
            q[products++] = g;
            continue;
        }
        const dim3 grid(static_cast<unsigned>(std::min<long long>((g.N + 255LL) / 256, 64)),
                        static_cast<unsigned>(std::min(g.M, 65535)));
        err = launch_early(g.dtype == kBf16 ? no_product_kernel<__nv_bfloat16> : no_product_kernel<__half>,
                           grid, 256, 0, stream, g);
        if (err != cudaSuccess) {
            *detail = "linear layer kernel launch failed";
            return err;
        }
    }
    // Aligned copies of the operands TMA cannot address, in one launch.
    PackJob jobs[2 * kMaxProducts] = {};
    const uint16_t **base[2 * kMaxProducts];
    size_t at[2 * kMaxProducts], elems = 0;
    int n_jobs = 0;
    auto pack = [&](const uint16_t *&ptr, long long &ld, int rows, int cols) {
        if (tma_rows(ptr, ld)) return;
        jobs[n_jobs] = pack_job(ptr, ld, rows, cols);
        base[n_jobs] = &ptr;
        at[n_jobs++] = elems;
        ld = (cols + 7LL) / 8 * 8;
        elems += static_cast<size_t>(rows) * ld;
    };
    for (int i = 0; i < products; ++i) {
        pack(q[i].A, q[i].lda, q[i].a_mn ? q[i].K : q[i].M, q[i].a_mn ? q[i].M : q[i].K);
        pack(q[i].B, q[i].ldb, q[i].b_mn ? q[i].K : q[i].N, q[i].b_mn ? q[i].N : q[i].K);
    }
    if (n_jobs > 0) {
        void *ptr = nullptr;
        err = layer_scratch(kScratchPack, stream, elems * 2, &ptr, detail);
        if (err != cudaSuccess) return err;
        for (int i = 0; i < n_jobs; ++i) {
            jobs[i].dst = static_cast<uint16_t *>(ptr) + at[i];
            *base[i] = jobs[i].dst;
        }
        for (int i = 0; i < n_jobs; i += 2) {
            const int blocks = jobs[i].gx * jobs[i].gy + jobs[i + 1].gx * jobs[i + 1].gy;
            err = launch_early(pack16_kernel, dim3(blocks), 256, 0, stream, jobs[i], jobs[i + 1]);
            if (err != cudaSuccess) {
                *detail = "repacking kernel launch failed";
                return err;
            }
        }
    }
    // Products that stream weights for a few rows go alone; the others share one launch (and a
    // gradient's two always do when there are more rows: 256 rows 1024 -> 1024 15.4 us, apart 22.5;
    // 4095 x 3001 x 1537 f16 108 us, apart 130).
    int together = 0;
    for (int i = 0; i < products; ++i) {
        if (stream_gemm16_supports(q[i]) && (n == 1 || q[i].M <= 64)) {
            err = stream_gemm16_launch(q[i], stream, detail);
            if (err != cudaSuccess) return err;
        } else {
            q[together++] = q[i];
        }
    }
    return together > 0 ? pair_gemm16_launch(q, together, stream, detail) : cudaSuccess;
}

cudaError_t act_grad_launch(const ActGrad &g, cudaStream_t stream, const char **detail) {
    cudaError_t err = cudaSuccess;
    if (g.M == 0) {
        err = launch_early(zero_kernel, dim3(static_cast<unsigned>((g.N + 255LL) / 256)), 256, 0, stream, g.db,
                           g.N);
    } else {
        const bool vec = g.N % 8 == 0 && tma_rows(g.dy, g.lddy) && (g.act == kActNone || tma_rows(g.z, g.ldz));
        // Rows per CTA, in whole steps: about whole rounds of the CTAs that run at once, three per SM, with 256
        // rows or so at most (a short last round) and a step at least (the last CTA of a column
        // block adds the sums of all of them). db alone, 2048 x 2048: 18.0 us with 8 rows, 9.5 with 32;
        // 4095 x 3001 unaligned: 49 us with 8 rows, 24.8 with 88 (1.2 rounds), 19.2 with 112 (one).
        const long long step = vec ? 32 : 16;  // rows that a CTA has under way at once
        const long long blocks = (g.N + static_cast<long long>(kGradCols) - 1) / kGradCols;
        int dev = 0, sms = 0;
        err = cudaGetDevice(&dev);
        if (err == cudaSuccess) err = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (err != cudaSuccess) {
            *detail = "device query failed";
            return err;
        }
        const long long resident = 3LL * sms;
        const long long rounds = g.M / std::max<long long>(1, resident / blocks) / 256 + 1;
        const long long want = std::max<long long>(1, rounds * resident / blocks);
        long long rows = std::max(step, (g.M / want + step / 2) / step * step);
        rows = std::max(rows, (g.M + 65534LL) / 65535);
        const int parts = static_cast<int>((g.M + rows - 1) / rows);
        float *part = nullptr;
        unsigned int *counters = nullptr;
        if (g.db && parts > 1) {
            void *p = nullptr, *q = nullptr;
            err = layer_scratch(kScratchSums, stream,
                                static_cast<size_t>(parts) * static_cast<size_t>(blocks) * kGradCols * 4, &p, detail);
            if (err == cudaSuccess)
                err = layer_scratch(kScratchSumSync, stream, static_cast<size_t>(blocks) * 4, &q, detail);
            if (err != cudaSuccess) return err;
            part = static_cast<float *>(p);
            counters = static_cast<unsigned int *>(q);
        }
        const dim3 grid(static_cast<unsigned>(blocks), static_cast<unsigned>(parts));
        auto kernel = g.dtype == kBf16
                          ? (vec ? act_grad_kernel<__nv_bfloat16, true> : act_grad_kernel<__nv_bfloat16, false>)
                          : (vec ? act_grad_kernel<__half, true> : act_grad_kernel<__half, false>);
        err = launch_early(kernel, grid, 256, 0, stream, g, static_cast<int>(rows), part, counters);
    }
    if (err != cudaSuccess) *detail = "gradient kernel launch failed";
    return err;
}

}  // namespace sg
