// moe16.cu: a whole mixture-of-experts layer for a few tokens on 16-bit values.
//
//   s_e = x . r_e;  p = softmax(s);  chosen: the k largest s_e, ties to the lowest e
//   w_j = p_chosen(j), divided by their sum when `renormalize`
//   h_j = act(G_e x) * (U_e x)   or, without a gate, act(U_e x)
//   y   = sum_j w_j D_e h_j + residual
//
// The fused kernel (moe_stream16.cu) takes layers whose matrices TMA can address; this file has the
// choice and the kernels for the others.
#include "activation16.cuh"
#include "half16.cuh"
#include "moe16.cuh"

#include <algorithm>

namespace sg {
namespace {

// One CTA per token: the scores (a warp per expert in turn), then the k largest and their
// weights by the first warp.
template <typename T>
__global__ void __launch_bounds__(256) moe_router_kernel(const Moe16 m, int *index, float *weight) {
    using H = Half16<T>;
    __shared__ float score[kMoeMaxExperts];
    const int t = blockIdx.x, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    if (m.active && !m.active[t]) {
        if (threadIdx.x < m.k) {
            index[t * m.k + threadIdx.x] = -1;
            weight[t * m.k + threadIdx.x] = 0.0f;
            if (m.index) m.index[t * m.k + threadIdx.x] = -1;
            if (m.weight) m.weight[t * m.k + threadIdx.x] = 0.0f;
        }
        return;
    }
    for (int e = w; e < m.E; e += 8) {
        float s = 0.0f;
        for (int i = lane; i < m.D; i += 32)
            s = fmaf(H::widen(m.X[t * m.ldx + i]), H::widen(m.Wr[e * m.ldr + i]), s);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (lane == 0) score[e] = s;
    }
    __syncthreads();
    if (w != 0) return;
    // Softmax statistics in fp32 over every expert; the largest is the first chosen one.
    float chosen[kMoeMaxTopk];
    unsigned long long below = ~0ull;
    float top = 0.0f;
    for (int j = 0; j < m.k; ++j) {
        unsigned long long best = 0;
        for (int e = lane; e < m.E; e += 32) {
            const unsigned long long key = moe_score_key(score[e], e);
            if (key < below && key > best) best = key;
        }
        for (int o = 16; o > 0; o >>= 1) best = max(best, __shfl_xor_sync(0xFFFFFFFFu, best, o));
        below = best;
        const int e = static_cast<int>(0xFFFFFFFFu - static_cast<unsigned>(best));
        if (j == 0) top = score[e];
        chosen[j] = expf(score[e] - top);
        if (lane == 0) {
            index[t * m.k + j] = e;
            if (m.index) m.index[t * m.k + j] = e;
        }
    }
    float sum = 0.0f;
    if (m.renormalize) {
        for (int j = 0; j < m.k; ++j) sum += chosen[j];
    } else {
        for (int e = lane; e < m.E; e += 32) sum += expf(score[e] - top);
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    }
    if (lane == 0)
        for (int j = 0; j < m.k; ++j) {
            weight[t * m.k + j] = chosen[j] / sum;
            if (m.weight) m.weight[t * m.k + j] = chosen[j] / sum;
        }
}

// ---- weights that TMA cannot address ----------------------------------------------------------------
//
// The products by fp32 FMAs: the rows are read as the aligned 4-byte words around them, 128 bytes
// per warp and instruction and several rows at once, against values of x (or h) in shared memory.
// Each (token, choice) reads its expert's weights; the choices of one expert run at the same time,
// so that memory sees them about once. 7 tokens, 4 experts of 1537 x 3001 bf16: 52 us (router 7, up 23,
// down 23) for 64 MB. (Loaders that bring such rows into the fused kernel's swizzled stages, through
// registers or cp.async, took 72 to 102 us: putting unaligned rows together costs more
// instructions than the two products here.)
constexpr int kSpan = 4096;  // values of x or h in shared memory at a time

// sum[r] += w_r[0 .. count) . x over this lane's words, ROWS rows at once.
template <typename T, int ROWS>
__device__ __forceinline__ void dot_rows(const uint16_t *const (&w)[ROWS], const float *x, int count, int lane,
                                         float (&sum)[ROWS]) {
    using H = Half16<T>;
    constexpr int UNROLL = 16 / ROWS;
    const uint32_t *p[ROWS];
    int shift[ROWS], words = 0;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(w[r]);
        p[r] = reinterpret_cast<const uint32_t *>(a & ~static_cast<uintptr_t>(3));
        shift[r] = static_cast<int>(a & 2u) >> 1;
        words = max(words, (count + shift[r] + 1) / 2);
    }
    for (int i0 = lane; i0 < words; i0 += 32 * UNROLL) {
        uint32_t v[UNROLL][ROWS];
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int r = 0; r < ROWS; ++r)
                if (2 * (i0 + 32 * u) - shift[r] < count) v[u][r] = __ldg(p[r] + i0 + 32 * u);
#pragma unroll
        for (int u = 0; u < UNROLL; ++u)
#pragma unroll
            for (int r = 0; r < ROWS; ++r) {
                const int at = 2 * (i0 + 32 * u) - shift[r];  // the word's first value
                if (at >= count) continue;
                const float2 f = H::widen2(v[u][r]);
                if (at >= 0) sum[r] = fmaf(f.x, x[at], sum[r]);
                if (at + 1 < count) sum[r] = fmaf(f.y, x[at + 1], sum[r]);
            }
    }
}

// Two hidden values f per warp (and their gates) of one (token, choice); h stays in fp32.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256) moe_up_kernel(const Moe16 m, const int *index, float *h) {
    using H = Half16<T>;
    __shared__ float x[kSpan];
    const int lane = threadIdx.x & 31;
    const int pair = blockIdx.y, t = pair / m.k, e = index[pair];
    if (e < 0) return;
    const int f = blockIdx.x * 16 + (threadIdx.x >> 5) * 2;
    constexpr int ROWS = GATED ? 4 : 2;
    float sum[ROWS] = {};
    for (int d0 = 0; d0 < m.D; d0 += kSpan) {
        const int count = min(kSpan, m.D - d0);
        __syncthreads();
        for (int i = threadIdx.x; i < count; i += 256) x[i] = H::widen(m.X[t * m.ldx + d0 + i]);
        __syncthreads();
        const uint16_t *w[ROWS];
#pragma unroll
        for (int r = 0; r < ROWS; ++r)  // a row past the last repeats it: its sum is not used
            w[r] = (r < 2 ? m.Wu : m.Wg) + e * m.su + min(f + (r & 1), m.F - 1) * m.ldu + d0;
        dot_rows<T, ROWS>(w, x, count, lane, sum);
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
        for (int o = 16; o > 0; o >>= 1) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], o);
    if (lane < 2 && f + lane < m.F) {
        const float u = lane ? sum[1] : sum[0], g = lane ? sum[ROWS - 1] : sum[ROWS - 2];
        float a = GATED ? g : u;
        with_activation(m.act, [&](auto act) { a = activate16<decltype(act)::value>(a); });
        h[pair * static_cast<long long>(m.F) + f + lane] = GATED ? a * u : a;
    }
}

// Four output values d per warp of one token: the choices in ascending j, then the residual.
template <typename T>
__global__ void __launch_bounds__(256) moe_down_kernel(const Moe16 m, const int *index,
                                                       const float *weight, const float *h) {
    using H = Half16<T>;
    __shared__ float x[kSpan];
    const int lane = threadIdx.x & 31, t = blockIdx.y;
    const int d = blockIdx.x * 32 + (threadIdx.x >> 5) * 4;
    float y[4] = {};
    for (int j = 0; j < m.k; ++j) {
        const int pair = t * m.k + j, e = index[pair];
        if (e < 0) continue;
        float sum[4] = {};
        for (int f0 = 0; f0 < m.F; f0 += kSpan) {
            const int count = min(kSpan, m.F - f0);
            __syncthreads();
            for (int i = threadIdx.x; i < count; i += 256) x[i] = h[pair * static_cast<long long>(m.F) + f0 + i];
            __syncthreads();
            const uint16_t *w[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) w[r] = m.Wd + e * m.sd + min(d + r, m.D - 1) * m.ldd + f0;
            dot_rows<T, 4>(w, x, count, lane, sum);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            for (int o = 16; o > 0; o >>= 1) sum[r] += __shfl_xor_sync(0xFFFFFFFFu, sum[r], o);
            y[r] = fmaf(weight[pair], sum[r], y[r]);
        }
    }
    if (lane < 4 && d + lane < m.D) {
        float v = lane == 0 ? y[0] : lane == 1 ? y[1] : lane == 2 ? y[2] : y[3];
        if (m.R) v += H::widen(m.R[t * m.ldres + d + lane]);
        m.Y[t * m.ldy + d + lane] = H::narrow(v);
    }
}

template <typename T>
cudaError_t launch(const Moe16 &m, cudaStream_t stream, const char **detail) {
    const size_t pairs = static_cast<size_t>(m.T) * m.k;
    void *p = nullptr;
    cudaError_t err = layer_scratch(kScratchMoe, stream, pairs * 8 + pairs * m.F * 4, &p, detail);
    if (err != cudaSuccess) return err;
    int *index = static_cast<int *>(p);
    float *weight = reinterpret_cast<float *>(index + pairs);
    float *h = weight + pairs;
    moe_router_kernel<T><<<m.T, 256, 0, stream>>>(m, index, weight);
    if (m.F > 0) {
        auto up = m.Wg ? moe_up_kernel<T, true> : moe_up_kernel<T, false>;
        up<<<dim3((m.F + 15LL) / 16, static_cast<unsigned>(pairs)), 256, 0, stream>>>(m, index, h);
    }
    if (m.D > 0)
        moe_down_kernel<T><<<dim3((m.D + 31LL) / 32, m.T), 256, 0, stream>>>(m, index, weight, h);
    err = cudaGetLastError();
    if (err != cudaSuccess) *detail = "mixture-of-experts kernel launch failed";
    return err;
}

}  // namespace

cudaError_t moe16_launch(const Moe16 &m, cudaStream_t stream, const char **detail) {
    if (moe_stream_supports(m)) return moe_stream_launch(m, stream, detail);
    return m.dtype == kBf16 ? launch<__nv_bfloat16>(m, stream, detail) : launch<__half>(m, stream, detail);
}

}  // namespace sg
