// checkpoint8.cu: 16-bit matrices to 8-bit checkpoints and back (checkpoint8.cuh has the form).
//
// Bound by memory: 2 + 1.06 bytes a value each way. A lane has 8 consecutive columns of a row, so that a
// block's maximum is three exchanges among 8 lanes; 8 to 32 lanes share a row, and a warp has several rows under
// way, so that its loads are out before the first is used.
#include "checkpoint8.cuh"
#include "layer16.cuh"

#include <algorithm>

namespace sg {
namespace {

constexpr int kRowsInFlight = 4;

// Lanes per row (8, 16 or 32) and the warps' tasks: 256 columns or less of kRowsInFlight steps of rows.
struct Split8 {
    int lanes, groups;  // groups: of 8 * lanes columns, per row
    long long row_tasks;
    __host__ __device__ int rows() const { return 32 / lanes * kRowsInFlight; }
};
Split8 split8(int M, long long chunks) {
    Split8 s;
    s.lanes = chunks <= 8 ? 8 : chunks <= 16 ? 16 : 32;
    s.groups = static_cast<int>((chunks + s.lanes - 1) / s.lanes);
    s.row_tasks = (M + s.rows() - 1LL) / s.rows();
    return s;
}
long long blocks8(const Split8 &s) { return (s.row_tasks * s.groups + 7) / 8; }

// VEC: X allows 16-byte loads (and N is a multiple of 8).
template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 5) save8_kernel(const Checkpoint8 c, const Split8 split, int q_vec) {
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31;
    const long long task = blockIdx.x * 8LL + (threadIdx.x >> 5);
    if (task >= split.row_tasks * split.groups) return;
    const long long row_task = task / split.groups;
    const int group = static_cast<int>(task - row_task * split.groups);
    const int step = 32 / split.lanes;
    const long long row0 = row_task * split.rows() + lane / split.lanes;
    const long long col = 8LL * (group * split.lanes + lane % split.lanes);
    const int count = static_cast<int>(max(0LL, min(8LL, c.N - col)));
    // Rows row0 + i * step with i < rows exist.
    const int rows = static_cast<int>(min(static_cast<long long>(kRowsInFlight), (c.M - row0 + step - 1) / step));
    constexpr int W = VEC ? 4 : 5;
    uint32_t raw[kRowsInFlight][W], top[kRowsInFlight];
    const uint16_t *src = c.X + row0 * c.ldx + col;
    const long long src_step = step * c.ldx;
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
#pragma unroll
        for (int k = 0; k < W; ++k) raw[i][k] = 0;
        if (i < rows && count > 0) {
            if constexpr (VEC) {
                const uint4 q = __ldg(reinterpret_cast<const uint4 *>(src + i * src_step));
                raw[i][0] = q.x;
                raw[i][1] = q.y;
                raw[i][2] = q.z;
                raw[i][3] = q.w;
            } else {
                load8_words(raw[i], src + i * src_step, count);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        if constexpr (!VEC) {
            const uint4 q = align8(raw[i], src + i * src_step);
            raw[i][0] = q.x;
            raw[i][1] = q.y;
            raw[i][2] = q.z;
            raw[i][3] = q.w;
            if (count < 8) {  // what follows the row is not part of it
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (2 * k >= count) raw[i][k] = 0;
                    if (2 * k + 1 == count) raw[i][k] &= 0xFFFFu;
                }
            }
        }
        top[i] = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) top[i] = magnitude2<T>(top[i], raw[i][k]);
        top[i] = magnitude(top[i]);
#pragma unroll
        for (int s = 1; s < 8; s *= 2) top[i] = max(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], s));
    }
    // Lane i of a block's eight has the scale of row i.
    const int mine = lane & 7;
    if (mine < rows && col / kCheckpointBlock * kCheckpointBlock < c.N) {
        uint32_t bits = top[0];
#pragma unroll
        for (int i = 1; i < kRowsInFlight; ++i) bits = mine == i ? top[i] : bits;
        c.S[(row0 + mine * step) * c.lds + col / kCheckpointBlock] = scale8<T>(bits);
    }
    if (count <= 0) return;
    int8_t *q = c.Q + row0 * c.ldq + col;
    const long long q_step = step * c.ldq;
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        if (i >= rows) break;
        const uint32_t w[4] = {raw[i][0], raw[i][1], raw[i][2], raw[i][3]};
        const uint2 codes = Coder8<T>(top[i]).eight(w);
        if (count == 8 && q_vec) {
            *reinterpret_cast<uint2 *>(q + i * q_step) = codes;
        } else {
            const uint64_t both = static_cast<uint64_t>(codes.y) << 32 | codes.x;
            for (int k = 0; k < count; ++k) q[i * q_step + k] = static_cast<int8_t>(both >> (8 * k));
        }
    }
}

// Aligned rows: X as VEC above, the codes in 8-byte words.
template <typename T>
__global__ void __launch_bounds__(256) restore8_aligned_kernel(const Restore8 c, const Split8 split) {
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31;
    const long long task = blockIdx.x * 8LL + (threadIdx.x >> 5);
    if (task >= split.row_tasks * split.groups) return;
    const long long row_task = task / split.groups;
    const int group = static_cast<int>(task - row_task * split.groups);
    const int step = 32 / split.lanes;
    const long long row0 = row_task * split.rows() + lane / split.lanes;
    const long long col = 8LL * (group * split.lanes + lane % split.lanes);
    if (col >= c.N || row0 >= c.M) return;
    const int rows = static_cast<int>(min(static_cast<long long>(kRowsInFlight), (c.M - row0 + step - 1) / step));
    const int8_t *q = c.Q + row0 * c.ldq + col;
    const float *s = c.S + row0 * c.lds + col / kCheckpointBlock;
    uint16_t *x = c.X + row0 * c.ldx + col;
    const long long q_step = step * c.ldq, s_step = step * c.lds, x_step = step * c.ldx;
    uint2 codes[kRowsInFlight];
    float scale[kRowsInFlight];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i)
        if (i < rows) {
            codes[i] = __ldg(reinterpret_cast<const uint2 *>(q + i * q_step));
            scale[i] = __ldg(s + i * s_step);
        }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i)
        if (i < rows) {
            const uint2 a = restore4<T>(codes[i].x, scale[i], scale[i], scale[i], scale[i]);
            const uint2 b = restore4<T>(codes[i].y, scale[i], scale[i], scale[i], scale[i]);
            *reinterpret_cast<uint4 *>(x + i * x_step) = make_uint4(a.x, a.y, b.x, b.y);
        }
}

// The output decides the alignment: a lane writes 16 aligned bytes of a row, and reads the codes of those
// columns, at any address, from the aligned 8-byte words that hold them. A row's first and last values are
// written one by one where they do not fill 16 bytes.
template <typename T>
__global__ void __launch_bounds__(256) restore8_kernel(const Restore8 c, const Split8 split) {
    grid_dependents();
    grid_dependency();
    const int lane = threadIdx.x & 31;
    const long long task = blockIdx.x * 8LL + (threadIdx.x >> 5);
    if (task >= split.row_tasks * split.groups) return;
    const long long row_task = task / split.groups;
    const int group = static_cast<int>(task - row_task * split.groups);
    const int step = 32 / split.lanes;
    const long long row0 = row_task * split.rows() + lane / split.lanes;
    const long long chunk = 8LL * (group * split.lanes + lane % split.lanes);
    uint64_t raw[kRowsInFlight][2];
    float scale[kRowsInFlight][2];
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        const long long row = row0 + i * step;
        raw[i][0] = raw[i][1] = 0;
        scale[i][0] = scale[i][1] = 0.0f;
        if (row >= c.M) continue;
        const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(c.X + row * c.ldx) >> 1) & 7;
        const long long first = max(0LL, chunk - shift), last = min(static_cast<long long>(c.N), chunk - shift + 8) - 1;
        if (first > last) continue;
        // Bytes first .. last lie in one or two aligned words.
        const uintptr_t at = reinterpret_cast<uintptr_t>(c.Q + row * c.ldq) + (chunk - shift);
        const uintptr_t word = at & ~static_cast<uintptr_t>(7);
        const uintptr_t lo = reinterpret_cast<uintptr_t>(c.Q + row * c.ldq + first);
        const uintptr_t hi = reinterpret_cast<uintptr_t>(c.Q + row * c.ldq + last);
        if (lo < word + 8) raw[i][0] = __ldg(reinterpret_cast<const unsigned long long *>(word));
        if (hi >= word + 8) raw[i][1] = __ldg(reinterpret_cast<const unsigned long long *>(word) + 1);
        const float *s = c.S + row * c.lds;
        scale[i][0] = __ldg(s + first / kCheckpointBlock);
        scale[i][1] = first / kCheckpointBlock == last / kCheckpointBlock ? scale[i][0] : __ldg(s + last / kCheckpointBlock);
    }
#pragma unroll
    for (int i = 0; i < kRowsInFlight; ++i) {
        const long long row = row0 + i * step;
        if (row >= c.M) continue;
        const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(c.X + row * c.ldx) >> 1) & 7;
        const long long col = chunk - shift;
        if (col >= c.N || col + 8 <= 0) continue;
        const int bytes = static_cast<int>(reinterpret_cast<uintptr_t>(c.Q + row * c.ldq) + col) & 7;
        const uint64_t both = bytes ? raw[i][0] >> (8 * bytes) | raw[i][1] << (64 - 8 * bytes) : raw[i][0];
        // Columns below `border` have the first scale.
        const int border = static_cast<int>((max(0LL, col) / kCheckpointBlock + 1) * kCheckpointBlock - col);
        auto of = [&](int k) { return k < border ? scale[i][0] : scale[i][1]; };
        const uint2 a = restore4<T>(static_cast<uint32_t>(both), of(0), of(1), of(2), of(3));
        const uint2 b = restore4<T>(static_cast<uint32_t>(both >> 32), of(4), of(5), of(6), of(7));
        uint16_t *x = c.X + row * c.ldx + col;
        if (col >= 0 && col + 8 <= c.N) {
            *reinterpret_cast<uint4 *>(x) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            const uint32_t v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k >= 0 && col + k < c.N) x[k] = static_cast<uint16_t>(v[k >> 1] >> (16 * (k & 1)));
        }
    }
}

}  // namespace

cudaError_t save8_launch(const Checkpoint8 &c, cudaStream_t stream, const char **detail) {
    const Split8 split = split8(c.M, (c.N + 7LL) / 8);
    const bool vec = tma_rows(c.X, c.ldx) && c.N % 8 == 0;
    const int q_vec = (reinterpret_cast<uintptr_t>(c.Q) & 7u) == 0 && c.ldq % 8 == 0;
    auto kernel = c.dtype == kBf16 ? (vec ? save8_kernel<__nv_bfloat16, true> : save8_kernel<__nv_bfloat16, false>)
                                   : (vec ? save8_kernel<__half, true> : save8_kernel<__half, false>);
    const cudaError_t err = blocks8(split) > 0x7fffffffLL
                                ? cudaErrorInvalidValue
                                : launch_early(kernel, dim3(static_cast<unsigned>(blocks8(split))), 256, 0, stream, c, split, q_vec);
    if (err != cudaSuccess) *detail = "checkpoint kernel launch failed";
    return err;
}

cudaError_t restore8_launch(const Restore8 &c, cudaStream_t stream, const char **detail) {
    const bool vec = tma_rows(c.X, c.ldx) && c.N % 8 == 0 && (reinterpret_cast<uintptr_t>(c.Q) & 7u) == 0 && c.ldq % 8 == 0;
    const Split8 split = split8(c.M, (c.N + (vec ? 7LL : 14LL)) / 8);  // a row may begin inside its first 16 bytes
    auto kernel = c.dtype == kBf16 ? (vec ? restore8_aligned_kernel<__nv_bfloat16> : restore8_kernel<__nv_bfloat16>)
                                   : (vec ? restore8_aligned_kernel<__half> : restore8_kernel<__half>);
    const cudaError_t err = blocks8(split) > 0x7fffffffLL
                                ? cudaErrorInvalidValue
                                : launch_early(kernel, dim3(static_cast<unsigned>(blocks8(split))), 256, 0, stream, c, split);
    if (err != cudaSuccess) *detail = "restore kernel launch failed";
    return err;
}

}  // namespace sg
