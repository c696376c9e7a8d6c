// pair_gemm16.cuh: the CTA-pair tensor-core product and the tensor maps of 16-bit matrices.
#pragma once

#include <cuda.h>
#include <math.h>

#include "layer16.cuh"

namespace sg {

// Tensor map of a rows x cols matrix of 16-bit values (cols contiguous, leading dimension ld),
// or, with depth > 0, of `depth` such matrices `stride` values apart; boxes of box_cols x box_rows
// with the 128-byte swizzle (narrow: 32 columns, the 64-byte one); values outside read as 0.
bool tensor_map_16(CUtensorMap *map, const void *base, int dtype, long long cols, long long rows,
                   long long ld, int box_cols, int box_rows, bool narrow = false, long long depth = 0,
                   long long stride = 0);
// Of a matrix of bytes, with the 64-byte swizzle.
bool tensor_map_8(CUtensorMap *map, const void *base, long long cols, long long rows, long long ld, int box_cols,
                  int box_rows);

// One grid over the tiles of one or two products (of two, the epilogue is the plain store: no
// bias, activation, residual or pre-activation). A and B must satisfy tma_rows; K > 0. The other
// matrices may have any alignment.
cudaError_t pair_gemm16_launch(const Gemm16 *list, int n, cudaStream_t stream, const char **detail);

// What the epilogue does with a product, besides Gemm16's own parts.
enum PairMode : int {  // (the streaming product has all but kPairSave8)
    kPairLayer = 0,  // bias, activation, residual, pre-activation
    kPairSave8,      // the same, the pre-activation as an 8-bit checkpoint
    kPairLogits,     // logits of the head: their sums of exponentials and the labels' values; no output
    kPairLogitGrad,  // the logits' gradient
    kPairSum,        // products that add to fp32 sums of earlier ones, and a factor from memory
};
struct PairSave8 {
    int8_t *codes = nullptr;
    long long ldq = 0;
    float *scales = nullptr;
    long long lds = 0;
};
// The k-blocks of 64 that one accumulator sums of the logits (see the pair product).
constexpr int kLogitBlocks = 16;
// The product's columns are the vocabulary's entries from v0 on.
struct PairHead {
    const int64_t *labels = nullptr;
    int V = 0, v0 = 0;
    int run = kLogitBlocks;  // of the streaming product, instead
    // kPairLogits: of 64 columns' logits z log2(e) of a row, the largest m and the sum of 2^(z log2(e) - m), at
    // parts[(column / 64) * ld_parts + row]; and the row's logit at its label. The streaming product: of
    // 32 columns' logits, at parts[row * ld_parts + column / 32].
    float2 *parts = nullptr;
    long long ld_parts = 0;
    float *at = nullptr;
    // kPairLogitGrad: the rows' weights are *factor * dloss, and the outputs are multiplied by 1 / *factor. Without a factor
    // all rows have one dloss: their weight is `unit`, and the outputs are multiplied by dloss; one that is not finite makes the
    // weight infinite or NaN, in the rows that count alone, and the outputs are left as they are.
    const float *lse = nullptr, *dloss = nullptr;
    long long incd = 0;
    const float *factor = nullptr;
    float unit = 1.0f;

    // Of row t, with f = *factor. (dloss is read per row in either case: with the row's lse, so that it costs no round trip
    // of its own.)
    __device__ __forceinline__ float weight(long long t, float f) const {
        const float d = dloss[t * incd];
        return factor ? f * d : fabsf(d) < INFINITY ? unit : unit * d;
    }
};
// The first product's sums, in the kernel's own order; a piece that is not the last writes no output.
struct PairSum {
    float *sums = nullptr;
    int first = 1, last = 1;
    const float *factor = nullptr;  // if finite, times scale, multiplies both products' outputs
    float scale = 1.0f;

    __device__ __forceinline__ float multiplier() const {
        const float f = *factor;
        return fabsf(f) < INFINITY ? scale * f : scale;
    }
};
struct PairExtra {
    PairSave8 save;
    PairHead head;
    PairSum sum;
};
size_t pair_sum_bytes(int M, int N);
cudaError_t pair_gemm16_extra_launch(const Gemm16 *list, int n, int mode, const PairExtra &extra,
                                     cudaStream_t stream, const char **detail);

// The product for few rows of A, streaming B's blocks once over all SMs: up to 64 rows, and more
// where the 128 x 64 tiles number at most 128. A and B must satisfy tma_rows; K > 0.
bool stream_gemm16_supports(const Gemm16 &g);
cudaError_t stream_gemm16_launch(const Gemm16 &g, cudaStream_t stream, const char **detail);
// kPairSum here: no sums, only the factor.
cudaError_t stream_gemm16_extra_launch(const Gemm16 &g, int mode, const PairExtra &extra, cudaStream_t stream,
                                       const char **detail);

}  // namespace sg
