// stream16.cuh: parts shared by the weight-streaming tensor-core kernels (a few tokens against
// large weights): the split of the work over CTAs, the shared-memory ring and the MMA loop.
//
// The product is computed transposed: a tile's 128 rows are 128 output features (weights are the
// MMA's A operand) and its NT columns are the tokens, so that every weight passes through shared
// memory once, whatever the number of tokens up to 256. The k-blocks of all tiles form one line
// of units, cut into equal runs, one per CTA (one CTA per SM): each SM streams the same number of
// bytes, however few tiles there are. A tile cut between CTAs is summed in fp32 from its pieces
// in the order of k, by the CTA whose piece arrives last (nothing waits).
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
        return static_cast<int>(((unit + 1LL) * ctas - 1) / total);
    }
};

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
