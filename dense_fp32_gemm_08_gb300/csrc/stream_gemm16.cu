// stream_gemm16.cu: D = act(A . B + bias) + res on 16-bit values for few rows of A (tokens), bound
// by streaming B (the weights) from memory once. The split of the work is in stream16.cuh. Roles
// of a CTA's warps:
//   warp 0, lane 0: TMA producer (a 128 x 64 block of weights and the tokens' 64 k values per unit)
//   warp 1, lane 0: MMA issuer into one of two TMEM accumulators of NT columns
//   warp 2:         TMEM allocation
//   warps 4..:      epilogue: lane = output feature, columns = 16 tokens per warp. Whole tiles go from
//                   TMEM to the epilogue; pieces go to scratch in fp32, and the warp that completes
//                   its part of a tile sums them in the order of k.
// Measured, one row 4096 -> 14336 bf16 with bias and SiLU (117 MB): 24.0 us, 4.9 TB/s: 112 whole tiles, of
// 64 blocks at 0.325 us, and 2.9 us until the first block arrives, for the epilogue and the launch. One row
// 14336 -> 16384 (470 MB): 77.9 us, 6.0 TB/s. 8 rows 512 -> 512: 5.0 us, launch and round trips to memory.
#include "activation16.cuh"
#include "layer16.cuh"
#include "pair_gemm16.cuh"
#include "stream16.cuh"

#include <algorithm>
#include <mutex>

namespace sg {
namespace {

constexpr int kMaxDevices = 64;
constexpr size_t kCounterBytes = 512 * 1024;  // arrival counters, up to 16 per tile

struct StreamParams {
    int M, N;  // tokens, output features
    int tiles, KB, m_tiles;  // tiles: of weights' rows x m_tiles of tokens, the tokens' running first
    UnitSplit split;
    uint32_t idesc;
    const uint16_t *bias;
    int act;
    const uint16_t *res;
    long long ldr;
    uint16_t *D;
    long long ldd;
    uint16_t *pre;
    long long ldz;
    unsigned int *counters;  // [tiles][epilogue warps], zero between calls
    float *pieces;           // [2 * CTAs][NT / 4][128][4]
};

template <int NT>
struct StreamConfig {
    static constexpr uint32_t A_BYTES = kStreamRows * kStreamK * 2;
    static constexpr uint32_t B_BYTES = NT * kStreamK * 2;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    // Four epilogue warps per 16 columns: their round trips to memory (pieces, outputs) overlap.
    static constexpr int GROUPS = NT / 16;
    static constexpr int THREADS = 128 + 128 * GROUPS;
    // Up to 32 tokens about 100 KiB of ring: enough in flight for the memory's full rate, and two CTAs
    // fit on an SM, so that the stream's next such kernel is resident, and its first weights on
    // their way to L2, while this one finishes (one token 4096 -> 14336: 26.2 -> 24.4 us).
    static constexpr bool TOKEN_TILES = NT == 64;  // fewer tokens are one tile
    static constexpr int CTAS = NT <= 32 ? 2 : 1;
    static constexpr int STAGES = NT <= 16 ? 6 : NT <= 32 ? 5 : 8;
    static constexpr uint32_t TMEM_COLS = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr size_t SMEM = STAGES * STAGE_BYTES + (2 * STAGES + 4) * 8 + 32 + 1024;
};

// 16 columns (tokens m0 .. m0 + 15) of output feature n.
template <typename T>
__device__ __forceinline__ void finish16(const StreamParams &p, int n, int m0, float b, float (&v)[16]) {
    using H = Half16<T>;
    if (n >= p.N) return;
    const int rows = min(16, p.M - m0);
    float r[16];
    if (p.res) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            r[i] = i < rows ? H::widen(p.res[(m0 + i) * p.ldr + n]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        v[i] += b;
        if (p.pre && i < rows) p.pre[(m0 + i) * p.ldz + n] = H::narrow(v[i]);
    }
    with_activation(p.act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 16; ++i) v[i] = activate16<decltype(a)::value>(v[i]);
    });
#pragma unroll
    for (int i = 0; i < 16; ++i)
        if (i < rows) p.D[(m0 + i) * p.ldd + n] = H::narrow(p.res ? v[i] + r[i] : v[i]);
}

template <int NT, bool W_MN, typename T>
__global__ void __launch_bounds__(StreamConfig<NT>::THREADS, StreamConfig<NT>::CTAS)
    stream_gemm16_kernel(const __grid_constant__ CUtensorMap map_w,
                         const __grid_constant__ CUtensorMap map_x, const StreamParams p) {
    using C = StreamConfig<NT>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + STAGES * C::STAGE_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;  // [2]
    uint64_t *acc_free = acc_full + 2;    // [2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int u0 = p.split.first(blockIdx.x), u1 = p.split.first(blockIdx.x + 1);

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_x);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&acc_full[j], 1);
            mbar_init(&acc_free[j], 4 * C::GROUPS);
        }
        mbar_init_fence();
    }
    if (warp == 2) tmem_alloc<1>(tmem_slot, C::TMEM_COLS);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    // The weights of the first stages go to L2 while the kernels before this one finish. (They are
    // read only after those have: L2 sees any write in between.)
    if (threadIdx.x == 0) {
        for (int u = u0; u < min(u1, u0 + STAGES); ++u) {
            const int tile = u / p.KB, kb = u - tile * p.KB, n0 = tile / p.m_tiles * kStreamRows;
            if (W_MN) {
                tma_prefetch_2d(&map_w, n0, kb * kStreamK);
                tma_prefetch_2d(&map_w, n0 + 64, kb * kStreamK);
            } else {
                tma_prefetch_2d(&map_w, kb * kStreamK, n0);
            }
        }
    }
    grid_dependency();

    if (warp == 0) {
        if (lane == 0) {
            RingCursor<STAGES> ring;
            int issued = 0;
            const int tile0 = u0 / p.KB;
            int kb = u0 - tile0 * p.KB, n0 = tile0 / p.m_tiles * kStreamRows, m0 = tile0 % p.m_tiles * NT;
            for (int u = u0; u < u1; ++u) {
                if (issued >= STAGES && !mbar_wait(&empty[ring.stage], ring.parity ^ 1u)) break;
                uint8_t *sw = smem + ring.stage * C::STAGE_BYTES, *sx = sw + C::A_BYTES;
                uint64_t *bar = &full[ring.stage];
                mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
                if (W_MN) {
                    tma_load_2d(sw, &map_w, bar, n0, kb * kStreamK);
                    tma_load_2d(sw + 8192, &map_w, bar, n0 + 64, kb * kStreamK);
                } else {
                    tma_load_2d(sw, &map_w, bar, kb * kStreamK, n0);
                }
                tma_load_2d(sx, &map_x, bar, kb * kStreamK, m0);
                ring.next();
                ++issued;
                if (++kb == p.KB) {
                    kb = 0;
                    m0 += NT;
                    if (m0 >= p.M) {
                        m0 = 0;
                        n0 += kStreamRows;
                    }
                }
            }
            grid_dependents();  // every copy is on its way: the next kernel may start its prologue
            // Shared memory must outlive every copy: wait (bounded) for the last stages.
            for (int j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
                if (!mbar_wait(&full[j % STAGES], (j / STAGES) & 1)) break;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            RingCursor<STAGES> ring;
            int j = -1, kb = u0 % p.KB;
            bool ok = true;
            uint32_t d = tmem;
            for (int u = u0; u < u1 && ok; ++u) {
                const bool first = u == u0 || kb == 0;
                if (first) {
                    ++j;
                    if (j >= 2 && !mbar_wait(&acc_free[j & 1], ((j >> 1) - 1) & 1)) break;
                    tc_after_sync();
                    d = tmem + static_cast<uint32_t>((j & 1) * NT);
                }
                if (!mbar_wait(&full[ring.stage], ring.parity)) break;
                tc_after_sync();
                const uint32_t sw = smem_addr(smem + ring.stage * C::STAGE_BYTES), sx = sw + C::A_BYTES;
                const uint64_t dw = W_MN ? desc_mn_major(sw, 8192) : desc_k_major(sw);
                const uint64_t dx = desc_k_major(sx);
#pragma unroll
                for (int k = 0; k < kStreamK / 16; ++k)
                    mma_16<1>(d, dw + static_cast<uint64_t>(k * (W_MN ? 128 : 2)),
                              dx + static_cast<uint64_t>(k * 2), p.idesc, !first || k > 0);
                mma_commit_16<1>(&empty[ring.stage]);
                ring.next();
                if (++kb == p.KB) kb = 0;
                if (kb == 0 || u + 1 == u1) mma_commit_16<1>(&acc_full[j & 1]);
            }
        }
    } else if (warp >= 4) {
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        constexpr int COLS = NT / C::GROUPS;
        const int first_col = (warp - 4) / 4 * COLS;
        int j = 0;
        for (int u = u0; u < u1; ++j) {
            const int tile = u / p.KB, kb0 = u - tile * p.KB;
            const int n_units = min(p.KB - kb0, u1 - u);
            u += n_units;
            const int n = (C::TOKEN_TILES ? tile / p.m_tiles : tile) * kStreamRows + row;
            const int m0 = C::TOKEN_TILES ? tile % p.m_tiles * NT : 0, tokens = min(NT, p.M - m0);
            const float b = p.bias && n < p.N ? Half16<T>::widen(p.bias[n]) : 0.0f;
            if (!mbar_wait(&acc_full[j & 1], (j >> 1) & 1)) break;
            tc_after_sync();
            const uint32_t acc = tmem + lane_base + static_cast<uint32_t>((j & 1) * NT);
            const bool whole = n_units == p.KB;
#pragma unroll 1
            for (int c = first_col; c < first_col + COLS; c += 16) {
                uint32_t r[16];
                tmem_ld_x16(acc + static_cast<uint32_t>(c), r);
                tmem_ld_wait();
                if (c + 16 == first_col + COLS) {
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[j & 1]);
                }
                if (c >= tokens) continue;
                if (whole) {
                    float v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
                    finish16<T>(p, n, m0 + c, b, v);
                } else {
                    put_piece<NT>(p.pieces, 2 * blockIdx.x + (kb0 == 0 ? 1 : 0), c, row, tokens, r);
                }
            }
            if (whole || first_col >= tokens ||
                !piece_arrived(p.counters + tile * 4 * C::GROUPS + warp - 4, n_units, p.KB, lane))
                continue;
            const int c0 = p.split.owner(tile * p.KB), c1 = p.split.owner(tile * p.KB + p.KB - 1);
#pragma unroll 1
            for (int c = first_col; c < min(tokens, first_col + COLS); c += 16) {
                float v[16];
                sum_pieces<NT>(p.pieces, c0, c1, 1, 0, c, row, tokens, v);
                finish16<T>(p, n, m0 + c, b, v);
            }
        }
    }

    __syncwarp();
    tc_before_sync();
    __syncthreads();
    if (warp == 2) {
        tc_after_sync();
        tmem_dealloc<1>(tmem, C::TMEM_COLS);
    }
}

template <int NT, bool W_MN, typename T>
cudaError_t launch(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    using C = StreamConfig<NT>;
    auto kernel = stream_gemm16_kernel<NT, W_MN, T>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        *detail = "cudaGetDevice failed";
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    }
    static std::once_flag once[kMaxDevices];
    static cudaError_t setup[kMaxDevices];
    static int sms[kMaxDevices];
    std::call_once(once[dev], [&] {
        setup[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(C::SMEM));
        if (setup[dev] == cudaSuccess)
            setup[dev] = cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev);
    });
    if (setup[dev] != cudaSuccess) {
        *detail = "linear layer kernel set-up failed";
        return setup[dev];
    }
    StreamParams p;
    p.M = g.M;
    p.N = g.N;
    p.m_tiles = (g.M + NT - 1) / NT;
    p.tiles = static_cast<int>((g.N + static_cast<long long>(kStreamRows) - 1) / kStreamRows) * p.m_tiles;
    p.KB = static_cast<int>((g.K + static_cast<long long>(kStreamK) - 1) / kStreamK);
    p.split.total = p.tiles * p.KB;
    // Equal pieces of every tile, of 5 blocks or more (8 for more columns, whose pieces take longer to
    // sum): a CTA then has one piece, and the tiles complete together. Else the blocks of all tiles in
    // equal runs over all SMs. Pieces where more would be shorter than that anyway, or where they take
    // less time: a block streams in 0.325 us on some of the SMs and 0.369 on all, whose rate memory
    // bounds; a whole tile takes 2.9 us besides, a cut one 4.4, runs that cross tiles 7.5. (One row,
    // pieces and runs: 96 tiles of 64 blocks 23.7 and 22.2 us, 112 23.9 and 24.9, 120 24.2 and 27.3; 112 of 224
    // blocks 76.0 and 69.1; 39 of 32 in three pieces 9.5 and 11.3; 52 of 224 in two 42.3 and 35.8.)
    const int by_blocks = std::max(1, p.KB / (NT == 16 ? 5 : 8));
    const int cut = std::min(by_blocks, sms[dev] / p.tiles);
    const double pieces_us = cut > 0 ? 0.325 * ((p.KB + cut - 1) / cut) + (cut > 1 ? 4.4 : 2.9) : 0.0;
    const double runs_us = 0.369 * p.split.total / sms[dev] + 7.5;
    if (cut > 0 && (cut == by_blocks || pieces_us < runs_us))
        p.split.ctas = p.tiles * cut;
    else
        p.split.ctas = std::min(sms[dev], std::max({1, p.split.total / min_run(NT), std::min(p.tiles, sms[dev])}));
    p.idesc = idesc_16(kStreamRows, NT, Half16<T>::kind, W_MN, false);
    p.bias = g.bias;
    p.act = g.act;
    p.res = g.res;
    p.ldr = g.ldr;
    p.D = g.D;
    p.ldd = g.ldd;
    p.pre = g.pre;
    p.ldz = g.ldz;
    void *ws = nullptr;
    err = layer_scratch(kScratchStream, stream,
                        kCounterBytes + static_cast<size_t>(2) * sms[dev] * 64 * kStreamRows * 4, &ws, detail);
    if (err != cudaSuccess) return err;
    p.counters = static_cast<unsigned int *>(ws);
    p.pieces = reinterpret_cast<float *>(static_cast<char *>(ws) + kCounterBytes);
    CUtensorMap mw, mx;
    if (!(W_MN ? tensor_map_16(&mw, g.B, g.dtype, g.N, g.K, g.ldb, 64, kStreamK)
               : tensor_map_16(&mw, g.B, g.dtype, g.K, g.N, g.ldb, kStreamK, kStreamRows)) ||
        !tensor_map_16(&mx, g.A, g.dtype, g.K, g.M, g.lda, kStreamK, NT)) {
        *detail = "cuTensorMapEncodeTiled rejected a matrix";
        return cudaErrorInvalidValue;
    }
    err = launch_early(kernel, dim3(p.split.ctas), C::THREADS, C::SMEM, stream, mw, mx, p);
    if (err != cudaSuccess) *detail = "linear layer kernel launch failed";
    return err;
}

template <int NT, typename T>
cudaError_t launch_major(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    return g.b_mn ? launch<NT, true, T>(g, stream, detail) : launch<NT, false, T>(g, stream, detail);
}

template <typename T>
cudaError_t launch_width(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    if (g.M <= 16) return launch_major<16, T>(g, stream, detail);
    if (g.M <= 32) return launch_major<32, T>(g, stream, detail);
    return launch_major<64, T>(g, stream, detail);
}

}  // namespace

// Up to 64 rows always. With more, the tiles here are 128 x 64 and a block of one takes 0.38 us on
// all SMs; the pair kernel's are 256 x 256 and take 0.30 us, one round of them up to 76. So this one
// wins while its tiles are fewer than 128 (256 rows 1024 -> 1024: 9.3 us here, 12.3 there; 128 rows
// 4096 -> 512: 12.5 and 26; 256 rows 4096 -> 4096, 128 tiles: 27.8 and 27.7; 512 rows: 45 and 28).
bool stream_gemm16_supports(const Gemm16 &g) {
    const long long m_tiles = (g.M + 63LL) / 64;
    const long long tiles = (g.N + static_cast<long long>(kStreamRows) - 1) / kStreamRows * m_tiles;
    const long long blocks = (g.K + static_cast<long long>(kStreamK) - 1) / kStreamK;
    return !g.a_mn && (g.M <= 64 || tiles <= 128) && tiles <= static_cast<long long>(kCounterBytes / 64) &&
           tiles * blocks <= 0x7fffffffLL;
}

cudaError_t stream_gemm16_launch(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    return g.dtype == kBf16 ? launch_width<__nv_bfloat16>(g, stream, detail)
                            : launch_width<__half>(g, stream, detail);
}

}  // namespace sg
