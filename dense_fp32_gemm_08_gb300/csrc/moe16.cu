// moe16.cu: a whole mixture-of-experts layer for a few tokens on 16-bit values.
//
//   s_e = x . r_e;  p = softmax(s);  chosen: the k largest s_e, ties to the lowest e
//   w_j = p_chosen(j), divided by their sum when `renormalize`
//   h_j = act(G_e x) * (U_e x)   or, without a gate, act(U_e x)
//   y   = sum_j w_j D_e h_j + residual
#include "epilogue.cuh"
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

// A warp per hidden value f of one (token, choice) pair; h stays in fp32.
template <typename T>
__global__ void __launch_bounds__(256) moe_up_kernel(const Moe16 m, const int *index, float *h) {
    using H = Half16<T>;
    const int lane = threadIdx.x & 31;
    const long long f = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int pair = blockIdx.y, t = pair / m.k, e = index[pair];
    if (f >= m.F || e < 0) return;
    const uint16_t *x = m.X + t * m.ldx;
    const uint16_t *u = m.Wu + e * m.su + f * m.ldu;
    const uint16_t *g = m.Wg ? m.Wg + e * m.su + f * m.ldu : nullptr;
    float su = 0.0f, sgate = 0.0f;
    for (int i = lane; i < m.D; i += 32) {
        const float xv = H::widen(x[i]);
        su = fmaf(xv, H::widen(u[i]), su);
        if (g) sgate = fmaf(xv, H::widen(g[i]), sgate);
    }
    for (int o = 16; o > 0; o >>= 1) {
        su += __shfl_xor_sync(0xFFFFFFFFu, su, o);
        sgate += __shfl_xor_sync(0xFFFFFFFFu, sgate, o);
    }
    if (lane == 0) h[pair * static_cast<long long>(m.F) + f] = g ? activate(sgate, m.act) * su : activate(su, m.act);
}

// A warp per output value d of one token: the choices in ascending j, then the residual.
template <typename T>
__global__ void __launch_bounds__(256) moe_down_kernel(const Moe16 m, const int *index,
                                                       const float *weight, const float *h) {
    using H = Half16<T>;
    const int lane = threadIdx.x & 31, t = blockIdx.y;
    const long long d = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    if (d >= m.D) return;
    float y = 0.0f;
    for (int j = 0; j < m.k; ++j) {
        const int pair = t * m.k + j, e = index[pair];
        if (e < 0) continue;
        const uint16_t *wd = m.Wd + e * m.sd + d * m.ldd;
        const float *hv = h + pair * static_cast<long long>(m.F);
        float s = 0.0f;
        for (int i = lane; i < m.F; i += 32) s = fmaf(hv[i], H::widen(wd[i]), s);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        y = fmaf(weight[pair], s, y);
    }
    if (lane == 0) {
        if (m.R) y += H::widen(m.R[t * m.ldres + d]);
        m.Y[t * m.ldy + d] = H::narrow(y);
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
    if (m.F > 0)
        moe_up_kernel<T><<<dim3((m.F + 7) / 8, static_cast<unsigned>(pairs)), 256, 0, stream>>>(m, index, h);
    if (m.D > 0)
        moe_down_kernel<T><<<dim3((m.D + 7) / 8, m.T), 256, 0, stream>>>(m, index, weight, h);
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
