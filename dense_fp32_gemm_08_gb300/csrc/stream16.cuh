// stream16.cuh: parts shared by the weight-streaming tensor-core kernels (a few tokens against
// large weights): the split of the work over CTAs, the shared-memory ring and the MMA loop.
//
// The product is computed transposed: a tile's 128 rows are 128 output features (weights are the
// MMA's A operand) and its NT columns are tokens, so that every weight passes through shared memory
// once for up to NT tokens. The k-blocks of all tiles form one line of units, cut into equal runs, one
// per CTA. There is a run for each SM at most, so that each streams the same number of bytes however
// few tiles there are, or as many runs as there are equal pieces of all tiles. A tile cut between
// CTAs is summed in fp32 from its pieces in the order of k, by the warp whose piece arrives last
// (nothing waits).
#pragma once

#include "tc16.cuh"

namespace sg {

constexpr int kStreamRows = 128;  // output features per tile
constexpr int kStreamK = 64;      // k values per block

// Units [first, last) of a CTA and the CTA that owns a unit.
struct UnitSplit {
    int total, ctas;
    __device__ __forceinline__ int first(int c) const {
        return static_cast<int>(static_cast<long long>(c) * total / ctas);
    }
    __device__ __forceinline__ int owner(int unit) const {
        const unsigned long long x = (unit + 1ull) * ctas - 1;
        if (x >> 32) return static_cast<int>(x / total);
        return static_cast<int>(static_cast<unsigned>(x) / static_cast<unsigned>(total));
    }
};

// A piece of a cut tile in scratch: fp32, four columns of a row together, the rows of a warp
// consecutive. Lane `row`'s address of columns 4 q .. 4 q + 3 in piece `slot`.
template <int NT>
__device__ __forceinline__ float4 *piece_at(float *pieces, int slot, int q, int row) {
    return reinterpret_cast<float4 *>(pieces) + (static_cast<size_t>(slot) * (NT / 4) + q) * kStreamRows + row;
}
// Columns c .. c + 15 of one row into / summed over pieces (in the order of k: the runs first ..
// last; a run that starts a tile keeps it in its odd slot). Only groups of four below `cols` exist.
template <int NT>
__device__ __forceinline__ void put_piece(float *pieces, int slot, int c, int row, int cols,
                                          const uint32_t (&r)[16]) {
#pragma unroll
    for (int g = 0; g < 4; ++g)
        if (c + 4 * g < cols)
            __stcg(piece_at<NT>(pieces, slot, c / 4 + g, row),
                   make_float4(__uint_as_float(r[4 * g]), __uint_as_float(r[4 * g + 1]),
                               __uint_as_float(r[4 * g + 2]), __uint_as_float(r[4 * g + 3])));
}
template <int NT>
__device__ __forceinline__ void sum_pieces(float *pieces, int first, int last, int stride, int offset, int c,
                                           int row, int cols, float (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = 0.0f;
#pragma unroll 4
    for (int k = first; k <= last; ++k) {  // the loads of four pieces are under way at once
        const int slot = (2 * k + (k == first ? 1 : 0)) * stride + offset;
#pragma unroll
        for (int g = 0; g < 4; ++g)
            if (c + 4 * g < cols) {
                const float4 q = __ldcg(piece_at<NT>(pieces, slot, c / 4 + g, row));
                v[4 * g] += q.x;
                v[4 * g + 1] += q.y;
                v[4 * g + 2] += q.z;
                v[4 * g + 3] += q.w;
            }
    }
}
// Counts `units` of a cut tile's part as arrived (a warp's 32 rows have their own counter); true
// for the warp that completes the tile's `total`, which then sees every piece.
__device__ __forceinline__ bool piece_arrived(unsigned int *counter, int units, int total, int lane) {
    __threadfence();
    __syncwarp();
    unsigned int done = 0;
    if (lane == 0) {
        __threadfence();
        done = atomicAdd(counter, static_cast<unsigned>(units)) + units;
        if (done == static_cast<unsigned>(total)) *counter = 0;  // for the next call
    }
    done = __shfl_sync(0xFFFFFFFFu, done, 0);
    if (done != static_cast<unsigned>(total)) return false;
    __threadfence();
    return true;
}
// Runs of fewer units would cut a tile into more pieces than summing them in turn is worth (a
// unit streams in about 0.1 us, a piece of 16 columns is summed in 0.2 us, of 64 in 0.8 us: equal runs
// over 8 rows 512 -> 512 take 5.0 us so, 6.4 with runs down to one unit).
__host__ __device__ constexpr int min_run(int nt) { return 8 + nt / 8; }

// Position in the ring, kept by each role across tiles and phases.
template <int STAGES>
struct RingCursor {
    int stage = 0;
    uint32_t parity = 0;
    __device__ __forceinline__ void next() {
        if (++stage == STAGES) {
            stage = 0;
            parity ^= 1u;
        }
    }
};

}  // namespace sg
