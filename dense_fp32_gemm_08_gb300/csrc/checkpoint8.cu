// checkpoint8.cu: 16-bit matrices to 8-bit checkpoints and back (checkpoint8.cuh has the form).
//
// Bound by memory: 2 + 1.06 bytes a value each way (16384 x 14336 bf16: saved in 102 us, 7.1 TB/s, restored in 103 us, 6.9
// TB/s; 4095 x 3001 in unaligned rows 10.6 and 10.4 us). Saving is near the issue rate too (65% of the cycles issue): a
// lane has 16 consecutive columns of a row, so that a block's maximum is two exchanges among 4 lanes and what a block costs
// besides its values is paid by 16 of them (with 8 columns: 137 us). Several rows are under way per lane, so that its
// loads are out before the first is used.
#include "checkpoint8.cuh"
#include "layer16.cuh"

#include <algorithm>

namespace sg {
namespace {

// Rows under way per lane. (16384 x 14336 saved with 2, 3, 4 at their best occupancy: 121, 111, 108 us, restored:
// 107, 103, 103 us. 4095 x 3001 in unaligned rows, saved: 11.3, 13.0, 12.7 us. All before the codes were made in paired
// operations, which the figures above have.)
__host__ __device__ constexpr int save_rows(bool vec) { return vec ? 4 : 2; }
constexpr int kRestoreRows = 4;

// A row's chunks of 16 (saving) or 8 columns over lanes (4, 8, 16 or 32 to a row), groups of 32 lanes over warps. A CTA's eight
// warps cover `wide` neighbouring groups (a power of two) of 8 / wide row tasks; a row task is
// as many steps of 32 / lanes rows as a lane has rows under way. (Powers of two: a division per task cost as much as its rows.)
struct Split8 {
    int lane_bits, wide_bits, groups, row_tasks;
    dim3 grid() const {
        return dim3(static_cast<unsigned>((groups + (1 << wide_bits) - 1) >> wide_bits),
                    static_cast<unsigned>(std::min((row_tasks + (8LL >> wide_bits) - 1) >> (3 - wide_bits), 65535LL)));
    }
};
Split8 split8(int M, long long chunks, int rows) {
    Split8 s;
    s.lane_bits = chunks <= 4 ? 2 : chunks <= 8 ? 3 : chunks <= 16 ? 4 : 5;
    s.groups = static_cast<int>((chunks + (1 << s.lane_bits) - 1) >> s.lane_bits);
    s.wide_bits = s.groups > 4 ? 3 : s.groups > 2 ? 2 : s.groups > 1 ? 1 : 0;
    s.row_tasks = static_cast<int>((M + (32LL >> s.lane_bits) * rows - 1) / ((32 >> s.lane_bits) * rows));
    return s;
}
// This warp's group and first row task, and how far apart its row tasks are.
struct Tasks8 {
    int group, task, apart;
    __device__ __forceinline__ explicit Tasks8(const Split8 &s) {
        const int warp = threadIdx.x >> 5;
        group = (blockIdx.x << s.wide_bits) + (warp & ((1 << s.wide_bits) - 1));
        task = (blockIdx.y << (3 - s.wide_bits)) + (warp >> s.wide_bits);
        apart = gridDim.y << (3 - s.wide_bits);
    }
};

// How many of the rows row0 + i * step, i < ROWS, exist.
template <int ROWS>
__device__ __forceinline__ int rows_left(int M, int row0, int step) {
    const long long left = static_cast<long long>(M) - row0;
    int rows = 0;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) rows += static_cast<long long>(i) * step < left;
    return rows;
}

// VEC: X allows 16-byte loads (and N is a multiple of 8). A lane has 16 columns of a row, four lanes a block.
template <typename T, bool VEC>
__device__ __forceinline__ void save8_rows(const Checkpoint8 &c, int lane, int row0, long long col, int step,
                                           bool q_vec) {
    constexpr int ROWS = save_rows(VEC);
    const int count = static_cast<int>(max(0LL, min(16LL, c.N - col)));
    const int rows = rows_left<ROWS>(c.M, row0, step);
    constexpr int W = VEC ? 4 : 5;
    uint32_t raw[ROWS][2][W], top[ROWS];
    const uint16_t *src = c.X + static_cast<long long>(row0) * c.ldx + col;
    const long long src_step = step * c.ldx;
#pragma unroll
    for (int i = 0; i < ROWS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int k = 0; k < W; ++k) raw[i][h][k] = 0;
            if (i < rows && count > 8 * h) {
                const uint16_t *p = src + i * src_step + 8 * h;
                if constexpr (VEC) {
                    const uint4 q = __ldg(reinterpret_cast<const uint4 *>(p));
                    raw[i][h][0] = q.x;
                    raw[i][h][1] = q.y;
                    raw[i][h][2] = q.z;
                    raw[i][h][3] = q.w;
                } else {
                    load8_words(raw[i][h], p, min(8, count - 8 * h));
                }
            }
        }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        top[i] = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if constexpr (!VEC) {
                const uint4 q = align8(raw[i][h], src + i * src_step + 8 * h);
                raw[i][h][0] = q.x;
                raw[i][h][1] = q.y;
                raw[i][h][2] = q.z;
                raw[i][h][3] = q.w;
                if (count < 8 * h + 8) {  // what follows the row is not part of it
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (8 * h + 2 * k >= count) raw[i][h][k] = 0;
                        if (8 * h + 2 * k + 1 == count) raw[i][h][k] &= 0xFFFFu;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) top[i] = magnitude2<T>(top[i], raw[i][h][k]);
        }
        top[i] = magnitude(top[i]);
#pragma unroll
        for (int s = 1; s < 4; s *= 2) top[i] = max(top[i], __shfl_xor_sync(0xFFFFFFFFu, top[i], s));
    }
    // Lane i of a block's four has the scale of row i.
    const int mine = lane & 3;
    if (mine < rows && col / kCheckpointBlock * kCheckpointBlock < c.N) {
        uint32_t bits = top[0];
#pragma unroll
        for (int i = 1; i < ROWS; ++i) bits = mine == i ? top[i] : bits;
        c.S[(static_cast<long long>(row0) + mine * step) * c.lds + col / kCheckpointBlock] = scale8<T>(bits);
    }
    if (count <= 0) return;
    int8_t *q = c.Q + static_cast<long long>(row0) * c.ldq + col;
    const long long q_step = step * c.ldq;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (i >= rows) break;
        const Coder8<T> coder(top[i]);
        uint2 codes[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w[4] = {raw[i][h][0], raw[i][h][1], raw[i][h][2], raw[i][h][3]};
            codes[h] = coder.eight(w);
        }
        if (count == 16 && q_vec) {
            *reinterpret_cast<uint4 *>(q + i * q_step) = make_uint4(codes[0].x, codes[0].y, codes[1].x, codes[1].y);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint64_t both = static_cast<uint64_t>(codes[h].y) << 32 | codes[h].x;
                for (int k = 0; k < min(8, count - 8 * h); ++k)
                    q[i * q_step + 8 * h + k] = static_cast<int8_t>(both >> (8 * k));
            }
        }
    }
}

// Aligned rows: 16-byte stores of X, the codes in 8-byte words. (A row's last word may hold bytes that follow it.)
// TAIL: N is not a multiple of 8. (One form for both restores 16384 x 14336 in 112 us, not 103.)
template <typename T, bool TAIL>
__device__ __forceinline__ void restore8_aligned_rows(const Restore8 &c, int row0, long long col, int step) {
    if (col >= c.N || row0 >= c.M) return;
    const int rows = rows_left<kRestoreRows>(c.M, row0, step);
    const int8_t *q = c.Q + static_cast<long long>(row0) * c.ldq + col;
    const float *s = c.S + static_cast<long long>(row0) * c.lds + col / kCheckpointBlock;
    uint16_t *x = c.X + static_cast<long long>(row0) * c.ldx + col;
    const long long q_step = step * c.ldq, s_step = step * c.lds, x_step = step * c.ldx;
    uint2 codes[kRestoreRows];
    float scale[kRestoreRows];
#pragma unroll
    for (int i = 0; i < kRestoreRows; ++i)
        if (i < rows) {
            codes[i] = __ldg(reinterpret_cast<const uint2 *>(q + i * q_step));
            scale[i] = __ldg(s + i * s_step);
        }
#pragma unroll
    for (int i = 0; i < kRestoreRows; ++i)
        if (i < rows) {
            const float2 s2 = make_float2(scale[i], scale[i]);
            const uint2 a = restore4<T>(codes[i].x, s2, s2), b = restore4<T>(codes[i].y, s2, s2);
            if (!TAIL || col + 8 <= c.N) {
                *reinterpret_cast<uint4 *>(x + i * x_step) = make_uint4(a.x, a.y, b.x, b.y);
            } else {
                const uint32_t v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
                for (int k = 0; k < 7; ++k)
                    if (col + k < c.N) x[i * x_step + k] = static_cast<uint16_t>(v[k >> 1] >> (16 * (k & 1)));
            }
        }
}

// The output decides the alignment: a lane writes 16 aligned bytes of a row, and reads the codes of those
// columns, at any address, from the aligned 8-byte words that hold them. A row's first and last values, where
// they do not fill 16 bytes, go one by one.
template <typename T>
__device__ __forceinline__ void restore8_any_rows(const Restore8 &c, int row0, long long chunk, int step) {
    uint2 raw[kRestoreRows][2];
    float scale[kRestoreRows][2];
    const int rows = rows_left<kRestoreRows>(c.M, row0, step);
    const int8_t *q = c.Q + static_cast<long long>(row0) * c.ldq;
    const float *s = c.S + static_cast<long long>(row0) * c.lds;
    uint16_t *x = c.X + static_cast<long long>(row0) * c.ldx;
    const long long q_step = step * c.ldq, s_step = step * c.lds, x_step = step * c.ldx;
    auto first_col = [&](int i) {
        return static_cast<int>(min(chunk, 0x7ffffff0LL)) - (static_cast<int>(reinterpret_cast<uintptr_t>(x + i * x_step) >> 1) & 7);
    };
    // Columns [first, last] of a chunk exist; a word is read where it holds the code of one of them.
#pragma unroll
    for (int i = 0; i < kRestoreRows; ++i) {
        const int col = first_col(i), first = max(col, 0), last = min(col + 7, c.N - 1);
        raw[i][0] = raw[i][1] = make_uint2(0, 0);
        scale[i][0] = scale[i][1] = 0.0f;
        if (i >= rows || first > last) continue;
        const int8_t *row = q + i * q_step;
        const uint2 *word = reinterpret_cast<const uint2 *>(reinterpret_cast<uintptr_t>(row + col) & ~static_cast<uintptr_t>(7));
        if (row + first < reinterpret_cast<const int8_t *>(word + 1)) raw[i][0] = __ldg(word);
        if (row + last >= reinterpret_cast<const int8_t *>(word + 1)) raw[i][1] = __ldg(word + 1);
        scale[i][0] = __ldg(s + i * s_step + first / kCheckpointBlock);
        scale[i][1] = __ldg(s + i * s_step + last / kCheckpointBlock);
    }
#pragma unroll
    for (int i = 0; i < kRestoreRows; ++i) {
        const int col = first_col(i);
        if (i >= rows || col >= c.N || col <= -8) continue;
        const int at = static_cast<int>(reinterpret_cast<uintptr_t>(q + i * q_step + col));
        const uint32_t w0 = at & 4 ? raw[i][0].y : raw[i][0].x, w1 = at & 4 ? raw[i][1].x : raw[i][0].y;
        const uint32_t w2 = at & 4 ? raw[i][1].y : raw[i][1].x;
        const uint32_t lo = __funnelshift_r(w0, w1, 8 * (at & 3)), hi = __funnelshift_r(w1, w2, 8 * (at & 3));
        const int border = (max(col, 0) / kCheckpointBlock + 1) * kCheckpointBlock - col;  // columns of the first scale
        auto of = [&](int k) { return k < border ? scale[i][0] : scale[i][1]; };
        auto two = [&](int k) { return make_float2(of(k), of(k + 1)); };
        const uint2 a = restore4<T>(lo, two(0), two(2)), b = restore4<T>(hi, two(4), two(6));
        uint16_t *to = x + i * x_step + col;
        if (col >= 0 && col <= c.N - 8) {
            *reinterpret_cast<uint4 *>(to) = make_uint4(a.x, a.y, b.x, b.y);
        } else {
            const uint32_t v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
            for (int k = 0; k < 8; ++k)
                if (col + k >= 0 && col + k < c.N) to[k] = static_cast<uint16_t>(v[k >> 1] >> (16 * (k & 1)));
        }
    }
}

// Calls body(lane, first row, chunk's first column, rows between a task's rows) for the warp's tasks. Row
// tasks past the last row keep their lanes together; their rows are left out by count.
template <int COLS, int ROWS, typename Body>
__device__ __forceinline__ void for_tasks(const Split8 &split, Body body) {
    const Tasks8 mine(split);
    if (mine.group >= split.groups) return;
    const int lane = threadIdx.x & 31, step = 32 >> split.lane_bits;
    const long long col = static_cast<long long>(COLS) * ((static_cast<long long>(mine.group) << split.lane_bits) + (lane & ((1 << split.lane_bits) - 1)));
    for (long long task = mine.task; task < split.row_tasks; task += mine.apart) {
        const long long row0 = task * ROWS * step + (lane >> split.lane_bits);
        body(lane, static_cast<int>(min(row0, 0x7fffffffLL)), col, step);
    }
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 4 : 5) save8_kernel(const Checkpoint8 c, const Split8 split, int q_vec) {
    grid_dependents();
    grid_dependency();
    for_tasks<16, save_rows(VEC)>(split, [&](int lane, int row0, long long col, int step) {
        save8_rows<T, VEC>(c, lane, row0, col, step, q_vec != 0);
    });
}
enum RestoreRows : int { kAnyRows, kAlignedRows, kAlignedTail };
template <typename T, int ROWS>
__global__ void __launch_bounds__(256) restore8_kernel(const Restore8 c, const Split8 split) {
    grid_dependents();
    grid_dependency();
    for_tasks<8, kRestoreRows>(split, [&](int, int row0, long long col, int step) {
        if constexpr (ROWS == kAnyRows)
            restore8_any_rows<T>(c, row0, col, step);
        else
            restore8_aligned_rows<T, ROWS == kAlignedTail>(c, row0, col, step);
    });
}

}  // namespace

cudaError_t save8_launch(const Checkpoint8 &c, cudaStream_t stream, const char **detail) {
    const bool vec = tma_rows(c.X, c.ldx) && c.N % 8 == 0;
    const Split8 split = split8(c.M, (c.N + 15LL) / 16, save_rows(vec));
    const int q_vec = (reinterpret_cast<uintptr_t>(c.Q) & 15u) == 0 && c.ldq % 16 == 0;
    auto kernel = c.dtype == kBf16 ? (vec ? save8_kernel<__nv_bfloat16, true> : save8_kernel<__nv_bfloat16, false>)
                                   : (vec ? save8_kernel<__half, true> : save8_kernel<__half, false>);
    const cudaError_t err = launch_early(kernel, split.grid(), 256, 0, stream, c, split, q_vec);
    if (err != cudaSuccess) *detail = "checkpoint kernel launch failed";
    return err;
}

cudaError_t restore8_launch(const Restore8 &c, cudaStream_t stream, const char **detail) {
    const bool vec = tma_rows(c.X, c.ldx) && (reinterpret_cast<uintptr_t>(c.Q) & 7u) == 0 && c.ldq % 8 == 0;
    const Split8 split = split8(c.M, (c.N + (vec ? 7LL : 14LL)) / 8, kRestoreRows);  // a row may begin inside its first 16 bytes
    auto choose = [&](auto type) {
        using T = decltype(type);
        return !vec ? restore8_kernel<T, kAnyRows> : c.N % 8 ? restore8_kernel<T, kAlignedTail> : restore8_kernel<T, kAlignedRows>;
    };
    auto kernel = c.dtype == kBf16 ? choose(__nv_bfloat16()) : choose(__half());
    const cudaError_t err = launch_early(kernel, split.grid(), 256, 0, stream, c, split);
    if (err != cudaSuccess) *detail = "restore kernel launch failed";
    return err;
}

}  // namespace sg
