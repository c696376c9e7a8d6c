// pair_gemm16.cuh: the CTA-pair tensor-core product and the tensor maps of 16-bit matrices.
#pragma once

#include <cuda.h>

#include "layer16.cuh"

namespace sg {

// Tensor map of a rows x cols matrix of 16-bit values (cols contiguous, leading dimension ld),
// or, with depth > 0, of `depth` such matrices `stride` values apart; boxes of box_cols x box_rows
// with the 128-byte swizzle (narrow: 32 columns, the 64-byte one); values outside read as 0.
bool tensor_map_16(CUtensorMap *map, const void *base, int dtype, long long cols, long long rows,
                   long long ld, int box_cols, int box_rows, bool narrow = false, long long depth = 0,
                   long long stride = 0);

// One grid over the tiles of one or two products (of two, the epilogue is the plain store: no
// bias, activation, residual or pre-activation). A and B must satisfy tma_rows; K > 0. The other
// matrices may have any alignment.
cudaError_t pair_gemm16_launch(const Gemm16 *list, int n, cudaStream_t stream, const char **detail);

// The product for few rows of A, streaming B's blocks once over all SMs: up to 64 rows, and more
// where the 128 x 64 tiles number at most 128. A and B must satisfy tma_rows; K > 0.
bool stream_gemm16_supports(const Gemm16 &g);
cudaError_t stream_gemm16_launch(const Gemm16 &g, cudaStream_t stream, const char **detail);

}  // namespace sg
