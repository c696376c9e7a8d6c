// head16.cu: the softmax cross entropy of a vocabulary head on 16-bit values, and its gradient,
// without keeping the logits z = X . op(W).
//
//   lse_t = log sum_v exp z_tv,   loss_t = lse_t - z_t,label
//   dz_tv = dloss_t (exp(z_tv - lse_t) - [v = label]),   dX = dz . op(W)^T,   dW = X^T . dz
//
// The forward pass is the pair product (pair_gemm16.cu) with an epilogue that reduces each row's 64
// logits of a warp to their maximum and sum of exponentials, or the streaming product for few tokens
// (stream_gemm16.cu) with one that does so for 32; a second kernel joins those. The gradient
// computes the logits again, a piece of the vocabulary at a time: one product whose epilogue
// writes the piece's dz in 16 bits to scratch, a pass over its entries at labels that are all but certain, then dX and
// dW's rows (or columns) of the piece in one launch. dX adds up over the pieces in fp32.
//
// Bound by the tensor cores for many tokens: 16384 of 32000 x 4096 bf16 2.24 to 2.45 ms for the loss (1,750 to 1,916
// TFLOP/s; the join 16 us of it), 6.47 to 7.12 ms for the gradient (three products, 1,810 to 1,990). For few by reading the
// weights: one token 48 us (5.5 TB/s). In between by the rounds of 256 x 256 tiles; unaligned weights are copied first (777
// tokens of 30001 x 1537 f16: 113 us, of which the copy is 29 and seven rounds of tiles for 6.2 are 75).
#include "activation16.cuh"
#include "half16.cuh"
#include "layer16.cuh"
#include "pair_gemm16.cuh"

#include <algorithm>

namespace sg {
namespace {

constexpr float kLn2 = 0.693147182f, kLn2Rest = -1.904654e-9f;  // ln 2 in two parts
// Maximum and sum of powers of 2 of two parts together. (A part of logits of -inf has m = -inf, s = 0. The maximum
// leaves NaN out, the sum does not: a part of NaN has m = -inf, s = NaN.)
__device__ __forceinline__ float2 join(float2 a, float2 b) {
    const float m = fmaxf(a.x, b.x);
    const float base = m == -INFINITY ? 0.0f : m;
    return make_float2(m, a.y * exp2_approx(a.x - base) + b.y * exp2_approx(b.x - base));
}
__device__ __forceinline__ float2 join_lanes(float2 a) {
#pragma unroll
    for (int s = 16; s > 0; s /= 2)
        a = join(a, make_float2(__shfl_xor_sync(0xFFFFFFFFu, a.x, s), __shfl_xor_sync(0xFFFFFFFFu, a.y, s)));
    return a;
}
// `n` parts, `apart` from one to the next, N loads of them under way at once.
template <int N>
__device__ __forceinline__ float2 join_run(const float2 *part, long long apart, int n) {
    float2 a = make_float2(-INFINITY, 0.0f);
    for (; n > 0; n -= N, part += N * apart) {
        float2 q[N];
#pragma unroll
        for (int k = 0; k < N; ++k) q[k] = k < n ? __ldcg(part + k * apart) : make_float2(-INFINITY, 0.0f);
        float m = a.x;
#pragma unroll
        for (int k = 0; k < N; ++k) m = fmaxf(m, q[k].x);
        const float base = m == -INFINITY ? 0.0f : m;
        float s = a.y * exp2_approx(a.x - base);
#pragma unroll
        for (int k = 0; k < N; ++k) s = fmaf(q[k].y, exp2_approx(q[k].x - base), s);
        a = make_float2(m, s);
    }
    return a;
}

// ---- labels that are all but certain --------------------------------------------------------------
//
// Where p is near 1 at the label, p - 1 has only the last digits of that one logit, and the accumulators of the
// tensor cores, which cut their sums, lose them: by up to a step of fp32 per 16 products (dX of such a token of 704 values
// 4e-2 off; 4e-3 in plain fp32). So those logits, and no others, are multiplied once more: x_t . w_label with
// every addition's rounding kept (Knuth's two-sum; products of 16-bit values are exact in fp32), within a step
// of fp32 of the true sum. The loss corrects lse and the label's logit with it, the gradient its dz there.
// It is done for 1 - p < 2^-6, in half 2^-3: above, what is lost is less than half a rounding of dz (logits of 10 in runs of
// 1024 lose 1.5e-5). (In the epilogues of the products, for every label, as it comes: 16384 tokens of 32000 x 4096 took
// 6% longer, of W stored D x V 3 times as long, of 56 entries 8 times.)
// Bound by reading rows of W, and columns 32 bytes per value where W is stored D x V. The loss and the gradient of 16384 tokens
// in ms, no label certain, and every one: V x D 32000 x 4096 2.28, 6.8, and 2.34, 6.9; stored D x V 2.28, 6.7, and 3.5, 7.8;
// 256 x 4096 stored D x V 0.034, 0.113, and 0.54, 0.31.
template <typename T>
constexpr float kCertain = Half16<T>::kind == kBf16 ? 0.015625f : 0.125f;  // 1 - p, and nearly -log p

struct LabelProduct {
    const uint16_t *x, *w;  // both in rows that TMA can address
    long long ldx, ldw;
    int D;
    bool w_dv;  // false: W stored V x D; true: D x V
};

struct KeptSum {
    float s = 0.0f, rest = 0.0f;
    __device__ __forceinline__ void add(float v) {
        const float t = s + v, b = t - s;  // b: what was added of v
        rest += (s - (t - b)) + (v - b);
        s = t;
    }
};

// Row `t` of X times row (D x V: column) `v` of W, by a whole warp; every lane has the result. UNROLL: loads of 8 values under
// way (D x V: 4 UNROLL of one).
template <typename T, int UNROLL>
__device__ __forceinline__ float label_logit(const LabelProduct &p, long long t, long long v, int lane) {
    using H = Half16<T>;
    KeptSum sum;
    const uint16_t *x = p.x + t * p.ldx;
    const unsigned D = p.D;  // (the last step may pass 2^31)
    if (p.w_dv) {
        const uint16_t *w = p.w + v;
        for (unsigned d0 = lane; d0 < D; d0 += 32 * 4 * UNROLL) {
            uint16_t xv[4 * UNROLL], wv[4 * UNROLL];
#pragma unroll
            for (int i = 0; i < 4 * UNROLL; ++i) {
                const unsigned d = d0 + 32 * i;
                xv[i] = d < D ? __ldg(x + d) : 0;
                wv[i] = d < D ? __ldg(w + d * p.ldw) : 0;
            }
#pragma unroll
            for (int i = 0; i < 4 * UNROLL; ++i) sum.add(__fmul_rn(H::widen(xv[i]), H::widen(wv[i])));
        }
    } else {
        const uint16_t *w = p.w + v * p.ldw;
        const unsigned whole = D & ~7u;
        for (unsigned d0 = 8 * lane; d0 < whole; d0 += 256 * UNROLL) {
            uint4 xv[UNROLL], wv[UNROLL];
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                xv[i] = wv[i] = make_uint4(0, 0, 0, 0);
                if (d0 + 256 * i < whole) {
                    xv[i] = __ldg(reinterpret_cast<const uint4 *>(x + d0 + 256 * i));
                    wv[i] = __ldg(reinterpret_cast<const uint4 *>(w + d0 + 256 * i));
                }
            }
#pragma unroll
            for (int i = 0; i < UNROLL; ++i) {
                const uint32_t a[4] = {xv[i].x, xv[i].y, xv[i].z, xv[i].w}, b[4] = {wv[i].x, wv[i].y, wv[i].z, wv[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 q = __fmul2_rn(H::widen2(a[k]), H::widen2(b[k]));
                    sum.add(q.x);
                    sum.add(q.y);
                }
            }
        }
        if (whole + lane < D) sum.add(__fmul_rn(H::widen(__ldg(x + whole + lane)), H::widen(__ldg(w + whole + lane))));
    }
#pragma unroll
    for (int m = 16; m > 0; m /= 2) {
        const float s = __shfl_xor_sync(0xFFFFFFFFu, sum.s, m);
        sum.rest += __shfl_xor_sync(0xFFFFFFFFu, sum.rest, m);
        sum.add(s);
    }
    return fabsf(sum.s) < INFINITY ? sum.s + sum.rest : sum.s;  // (the roundings of an infinite sum are NaN)
}

struct LossOut {
    const float *at;
    const int64_t *labels;
    int T, V;
    float *loss, *lse;
    LabelProduct product;
    // By a whole warp, each lane with the row's `a`.
    template <typename T16, int UNROLL>
    __device__ __forceinline__ void put(int row, float2 a, int lane) const {
        const float l = a.x == -INFINITY && a.y == 0.0f ? a.x : fmaf(a.x, kLn2, fmaf(a.x, kLn2Rest, logf(a.y)));
        const int64_t label = labels[row];
        const bool counts = label >= 0 && label < V;
        const float minus_logp = counts ? l - at[row] : 0.0f;
        if (counts && minus_logp < kCertain<T16>) {
            put_certain<T16, UNROLL>(row, l, lane);
        } else if (lane == 0) {
            if (lse) lse[row] = l;
            if (loss) loss[row] = minus_logp;
        }
    }
    // (Not part of the joins' code: its registers made theirs spill.)
    template <typename T16, int UNROLL>
    __device__ __noinline__ void put_certain(int row, float l, int lane) const {
        const float z = at[row], exact = label_logit<T16, UNROLL>(product, row, labels[row], lane);
        if (lane != 0) return;
        // The sum's share of it changes by that difference, which is small; and no sum is below one of its parts.
        l = fmaxf(fmaf(expf(z - l), exact - z, l), exact);
        if (lse) lse[row] = l;
        if (loss) loss[row] = l - exact;
    }
};

// Joins the parts of 32 rows, parts[part][row]: lane = row, a warp every 32nd part, then the warps through
// shared memory. (500 parts of 16384 rows 16 us, of 777 rows 6 us.)
constexpr int kJoinThreads = 1024;
template <typename T16>
__global__ void __launch_bounds__(kJoinThreads, 2) join_kernel(const float2 *parts, long long ld, int n_parts,
                                                            const __grid_constant__ LossOut out) {
    __shared__ float2 shared[32][33];
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = blockIdx.x * 32 + lane;
    float2 a = make_float2(-INFINITY, 0.0f);
    if (row < out.T) a = join_run<6>(parts + warp * ld + row, 32 * ld, (n_parts - warp + 31) / 32);
    shared[warp][lane] = a;
    __syncthreads();
    // Warp w now joins row w's 32 values.
    a = join_lanes(shared[lane][warp]);
    const int mine = blockIdx.x * 32 + warp;
    if (mine < out.T) out.put<T16, 1>(mine, a, lane);
}

// Joins parts[row][part]: a row per warp, or per CTA where it has many parts.
constexpr int kRowWarps = 8;
template <typename T16>
__global__ void __launch_bounds__(32 * kRowWarps) join_rows_kernel(const float2 *parts, long long ld, int n_parts,
                                                                   int wide, const __grid_constant__ LossOut out) {
    __shared__ float2 shared[kRowWarps];
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = wide ? blockIdx.x : blockIdx.x * kRowWarps + warp;
    float2 a = make_float2(-INFINITY, 0.0f);
    if (row < out.T) {
        const int first = wide ? threadIdx.x : lane, step = wide ? 32 * kRowWarps : 32;
        a = join_run<4>(parts + row * ld + first, step, (n_parts - first + step - 1) / step);
    }
    a = join_lanes(a);
    if (!wide) {
        if (row < out.T) out.put<T16, 4>(row, a, lane);
        return;
    }
    if (lane == 0) shared[warp] = a;
    __syncthreads();
    if (warp == 0) {
        a = join_lanes(lane < kRowWarps ? shared[lane] : make_float2(-INFINITY, 0.0f));
        out.put<T16, 4>(row, a, lane);
    }
}

// The products of the gradient read dz in 16 bits. It is stored for rows' weights of `unit` at most, dloss
// over its largest magnitude m, and the outputs are multiplied by m / unit: where every token has the same
// dloss (a mean), dz is then p - [v = label] itself, which near -1 is rounded with almost no error, where a
// dloss between powers of two would round all rows the same way. In half, whose smallest value is 2^-24, unit =
// 2^14 keeps probabilities down to 2^-38.
float unit_of(int dtype) { return dtype == kF16 ? 16384.0f : 1.0f; }

// factor[0] = unit / m, factor[1] = m, with m the largest finite |dloss| of the counted tokens.
__global__ void __launch_bounds__(1024) factor_kernel(const float *dloss, long long incd, const int64_t *labels,
                                                      int T, int V, float unit, float *factor) {
    __shared__ float top[32];
    grid_dependents();
    grid_dependency();
    float a = 0.0f;
#pragma unroll 4
    for (long long t = threadIdx.x; t < T; t += 1024) {
        const int64_t label = labels[t];
        const float d = fabsf(dloss[t * incd]);
        if (label >= 0 && label < V && d < INFINITY) a = fmaxf(a, d);
    }
#pragma unroll
    for (int s = 16; s > 0; s /= 2) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, s));
    if ((threadIdx.x & 31) == 0) top[threadIdx.x >> 5] = a;
    __syncthreads();
    if (threadIdx.x < 32) {
        a = top[threadIdx.x];
#pragma unroll
        for (int s = 16; s > 0; s /= 2) a = fmaxf(a, __shfl_xor_sync(0xFFFFFFFFu, a, s));
        if (threadIdx.x == 0) {
            a = a > 0.0f ? fmaxf(a, 1e-30f) : 1.0f;
            factor[0] = unit / a;
            factor[1] = a;
        }
    }
}

// The entries of dz at labels that are all but certain once more, of a piece of n entries: a warp finds them among
// `each` tokens, as few as fill the GPU once (32 at most), and multiplies them one by one. (1.3 to 4 us of the gradient, and
// 1 to 2.5 more for few tokens where there are such labels. With runs of 64 on the streaming product in place of it: 16 tokens
// of 32000 x 4096 168.5 us and 163.5, 256 of 1000 x 512 f16 18.3 and 18.5, with such labels 18.2 and 19.8; dX of one
// token of 56 x 704 up to 2.7e-2 off and 7.1e-3, in plain fp32 7.8e-3.)
int tokens_each(int T) { return std::min(32, 1 + T / 8192); }
template <typename T16>
__global__ void __launch_bounds__(256) certain_kernel(const PairHead h, const LabelProduct product, uint16_t *dz, long long ldz,
                                                      int T, int n, int each) {
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31;
    const long long t0 = (blockIdx.x * 8LL + (threadIdx.x >> 5)) * each, t = t0 + lane;
    long long label = -1;  // of the entries from v0 on
    float lse = 0.0f, weight = 0.0f;
    bool certain = false;
    if (lane < each && t < T) {
        const int64_t l = h.labels[t];
        lse = h.lse[t];
        weight = h.weight(t, h.factor ? *h.factor : 1.0f);
        if (l >= h.v0 && l - h.v0 < n) {
            label = l - h.v0;
            // weight (p - 1); a weight or value that is not finite is not among them
            certain = fabsf(Half16<T16>::widen(dz[t * ldz + label])) < kCertain<T16> * fabsf(weight);
        }
    }
    for (unsigned todo = __ballot_sync(0xFFFFFFFFu, certain); todo != 0; todo &= todo - 1) {
        const int i = __ffs(todo) - 1;
        const float z = label_logit<T16, 4>(product, t0 + i, __shfl_sync(0xFFFFFFFFu, label, i), lane);
        if (lane == i) dz[t * ldz + label] = Half16<T16>::narrow(weight * expm1f(z - lse));
    }
}

// The logits of tokens [t0, t0 + T) and vocabulary entries [v0, v0 + n).
Gemm16 logits(const Head16 &h, int t0, int T, int v0, int n) {
    Gemm16 g;
    g.dtype = h.dtype;
    g.M = T;
    g.N = n;
    g.K = h.D;
    g.A = h.X + static_cast<long long>(t0) * h.ldx;
    g.lda = h.ldx;
    g.B = h.w_dv ? h.W + v0 : h.W + static_cast<long long>(v0) * h.ldw;
    g.ldb = h.ldw;
    g.b_mn = h.w_dv;
    return g;
}

LabelProduct label_product(const Gemm16 &g) { return {g.A, g.B, g.lda, g.ldb, g.K, g.b_mn}; }

// k-blocks that one accumulator of the streaming product sums: runs of 512 values, and of 64 in the loss of at most 512
// entries. (The loss in us: one token of 32000 x 4096 47.8 and 52.4, 7899 of 48 x 1816 18.6 and 22.4.)
constexpr int kGradRun = 8;
int loss_run(const Head16 &h) { return h.V <= 512 ? 1 : kGradRun; }

cudaError_t pack(Head16 &h, cudaStream_t stream, const char **detail) {
    const Pack16 packs[2] = {{&h.X, &h.ldx, h.T, h.D}, {&h.W, &h.ldw, h.w_dv ? h.D : h.V, h.w_dv ? h.V : h.D}};
    return pack16_launch(packs, 2, stream, detail);
}

constexpr int kTokens = 32768;  // per piece of the forward pass: 131072 entries then leave 0.5 GB of parts

}  // namespace

cudaError_t head16_launch(const Head16 &head, cudaStream_t stream, const char **detail) {
    Head16 h = head;
    cudaError_t err = pack(h, stream, detail);
    if (err != cudaSuccess) return err;
    for (int t0 = 0; t0 < h.T; t0 += std::min(kTokens, h.T - t0)) {
        const int T = std::min(kTokens, h.T - t0);
        const Gemm16 g = logits(h, t0, T, 0, h.V);
        const bool few = stream_gemm16_supports(g);
        const int n_parts = static_cast<int>((h.V + (few ? 31LL : 63LL)) / (few ? 32 : 64));
        const long long ld = (T + 31LL) / 32 * 32, ld_parts = few ? n_parts : ld;
        void *p = nullptr;
        err = layer_scratch(kScratchHead, stream,
                            static_cast<size_t>(ld) * 4 + static_cast<size_t>(few ? T : ld) * n_parts * 8, &p, detail);
        if (err != cudaSuccess) return err;
        PairExtra extra;
        PairHead &x = extra.head;
        x.labels = h.labels + t0;
        x.V = h.V;
        x.run = loss_run(h);
        x.at = static_cast<float *>(p);
        x.parts = reinterpret_cast<float2 *>(x.at + ld);
        x.ld_parts = ld_parts;
        const LossOut out{x.at, x.labels, T, h.V, h.loss ? h.loss + t0 : nullptr, h.lse ? h.lse + t0 : nullptr,
                          label_product(g)};
        const float2 *parts = x.parts;
        if (few) {
            err = stream_gemm16_extra_launch(g, kPairLogits, extra, stream, detail);
            if (err != cudaSuccess) return err;
            const int wide = n_parts > 128;
            err = launch_early(h.dtype == kBf16 ? join_rows_kernel<__nv_bfloat16> : join_rows_kernel<__half>,
                               dim3(static_cast<unsigned>(wide ? T : (T + kRowWarps - 1) / kRowWarps)), 32 * kRowWarps, 0,
                               stream, parts, ld_parts, n_parts, wide, out);
        } else {
            err = pair_gemm16_extra_launch(&g, 1, kPairLogits, extra, stream, detail);
            if (err != cudaSuccess) return err;
            err = launch_early(h.dtype == kBf16 ? join_kernel<__nv_bfloat16> : join_kernel<__half>,
                               dim3(static_cast<unsigned>((T + 31) / 32)), kJoinThreads, 0, stream, parts, ld_parts, n_parts, out);
        }
        if (err != cudaSuccess) {
            *detail = "loss kernel launch failed";
            return err;
        }
    }
    return cudaSuccess;
}

cudaError_t head16_grad_launch(const Head16 &head, cudaStream_t stream, const char **detail) {
    Head16 h = head;
    cudaError_t err = pack(h, stream, detail);
    if (err != cudaSuccess) return err;
    // Pieces of up to 512 MB of dz, of 4096 entries or more, all of about the same size: each one's dX passes through
    // memory in fp32. (16384 tokens of 32000 x 4096 with 128, 256, 512, 1024 MB: 7.21, 6.94, 6.73, 6.79 ms; 8192 of
    // 65536 x 1024: 2.08, 1.96, 1.92, 1.92.)
    const long long most = std::max<long long>(4096, (512LL << 20) / 2 / h.T / 256 * 256);
    const long long pieces = (h.V + most - 1) / most;
    const long long width = ((h.V + pieces - 1) / pieces + 255) / 256 * 256;
    const long long ldz = std::min(width, (h.V + 7LL) / 8 * 8);
    void *dz = nullptr, *p = nullptr;
    err = layer_scratch(kScratchHeadDz, stream, static_cast<size_t>(h.T) * ldz * 2, &dz, detail);
    if (err != cudaSuccess) return err;
    PairExtra extra;
    PairHead &x = extra.head;
    x.labels = h.labels;
    x.V = h.V;
    x.run = kGradRun;
    x.lse = h.lse_in;
    x.dloss = h.dloss;
    x.incd = h.incd;
    const float unit = unit_of(h.dtype);
    extra.sum.scale = 1.0f / unit;
    x.unit = unit;
    if (h.incd == 0) {
        extra.sum.factor = h.dloss;
    } else {
        err = layer_scratch(kScratchHead, stream, 8, &p, detail);
        if (err != cudaSuccess) return err;
        float *factor = static_cast<float *>(p);
        err = launch_early(factor_kernel, dim3(1), 1024, 0, stream, h.dloss, h.incd, h.labels, h.T, h.V, unit, factor);
        if (err != cudaSuccess) {
            *detail = "loss gradient kernel launch failed";
            return err;
        }
        x.factor = factor;
        extra.sum.factor = factor + 1;
    }
    if (h.dX && width < h.V) {
        err = layer_scratch(kScratchHeadSum, stream, pair_sum_bytes(h.T, h.D), &p, detail);
        if (err != cudaSuccess) return err;
        extra.sum.sums = static_cast<float *>(p);
    }
    for (long long next = 0; next < h.V; next += width) {
        const int v0 = static_cast<int>(next), n = static_cast<int>(std::min<long long>(width, h.V - next));
        Gemm16 g = logits(h, 0, h.T, v0, n);
        g.D = static_cast<uint16_t *>(dz);
        g.ldd = ldz;
        x.v0 = v0;
        err = stream_gemm16_supports(g) ? stream_gemm16_extra_launch(g, kPairLogitGrad, extra, stream, detail)
                                        : pair_gemm16_extra_launch(&g, 1, kPairLogitGrad, extra, stream, detail);
        if (err != cudaSuccess) return err;
        const int each = tokens_each(h.T);
        err = launch_early(h.dtype == kBf16 ? certain_kernel<__nv_bfloat16> : certain_kernel<__half>,
                           dim3(static_cast<unsigned>((h.T + 8LL * each - 1) / (8 * each))), 256, 0, stream, x,
                           label_product(g), g.D, ldz, h.T, n, each);
        if (err != cudaSuccess) {
            *detail = "loss gradient kernel launch failed";
            return err;
        }
        Gemm16 list[2];
        int count = 0;
        if (h.dX) {
            Gemm16 &q = list[count++];
            q.dtype = h.dtype;
            q.M = h.T;
            q.N = h.D;
            q.K = n;
            q.A = g.D;
            q.lda = ldz;
            q.B = g.B;
            q.ldb = h.ldw;
            q.b_mn = !h.w_dv;
            q.D = h.dX;
            q.ldd = h.lddx;
            // Up to 64 tokens and from 2048 entries on, dX streams the weights by itself; else it is in one grid
            // with dW. (1 token, apart and together: 1000 x 512 16.6 and 12.4 us, 2000 x 512 17.0 and 17.6, 4000 x 512
            // 17.7 and 22.9. 64 tokens: 1000 x 1024 24.0 and 19.0, 2000 x 1024 24.0 and 24.3, 8000 x 256 22.4 and 31.3.)
            if (h.T <= 64 && n == h.V && n >= 2048 && stream_gemm16_supports(q)) {
                err = stream_gemm16_extra_launch(q, kPairSum, extra, stream, detail);
                if (err != cudaSuccess) return err;
                --count;
            }
        }
        if (h.dW) {
            Gemm16 &q = list[count++];
            q.dtype = h.dtype;
            q.M = h.w_dv ? h.D : n;
            q.N = h.w_dv ? n : h.D;
            q.K = h.T;
            q.A = h.w_dv ? h.X : g.D;
            q.lda = h.w_dv ? h.ldx : ldz;
            q.a_mn = true;
            q.B = h.w_dv ? g.D : h.X;
            q.ldb = h.w_dv ? ldz : h.ldx;
            q.b_mn = true;
            q.D = h.w_dv ? h.dW + v0 : h.dW + static_cast<long long>(v0) * h.lddw;
            q.ldd = h.lddw;
        }
        extra.sum.first = v0 == 0;
        extra.sum.last = v0 + n == h.V;
        if (count > 0) err = pair_gemm16_extra_launch(list, count, kPairSum, extra, stream, detail);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace sg
