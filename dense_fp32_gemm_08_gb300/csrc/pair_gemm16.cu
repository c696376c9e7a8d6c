// pair_gemm16.cu: D = act(A . B + bias) + res on 16-bit values with tcgen05 MMAs over pairs of
// CTAs (cta_group::2): one MMA multiplies 256 rows by 256 columns, each CTA of the pair holding
// half of A's rows and half of B's columns in its own shared memory, so each SM stages half the
// operand bytes per multiply-add of a one-CTA tile. (Narrower tiles, 128 to 192 columns, took about as
// long per k-block as 256, 0.30 us: a stage's way from L2 bounds them. 224 gained 1 to 3% where
// the rounds of tiles stay the same and lost 7% on large products.)
//
// A persistent grid of pairs walks the output tiles of one product, or of the two of a gradient
// one after the other (the idle part of a last round is then paid once), in grouped-raster order.
// A product with few tiles and a long k (a weight gradient over many rows) has its tiles cut along
// k: the pieces go to scratch in fp32, and each epilogue warp that finds its 32 x 64 values complete
// (a count in memory; nothing waits) sums them in the order of k.
// Roles of a CTA's 20 warps:
//   warp 0, lane 0: TMA producer: this CTA's 128 rows of A and 128 columns of B per 64-wide
//                   k-block into a ring of 6 stages (512 x 12288 x 4096 with 4, 5, 6: 55, 49.3 and
//                   47.5 us, so the sixth has the room of a second store buffer per epilogue warp);
//                   both CTAs' copies complete on the leader's "full" barrier.
//   warp 1, lane 0: (leader CTA) issues the MMAs, four k-steps of 16 per block, into one of two
//                   TMEM accumulators of 256 columns; commits free the stage in both CTAs and,
//                   at a tile's end, hand the accumulator to both CTAs' epilogues.
//   warp 2:         allocates and frees the pair's TMEM.
//   warps 4..19:    epilogue of this CTA's 128 rows while the next tile multiplies: warp w has TMEM
//                   lanes 32 (w % 4) .. + 31 and 64 of the columns, 32 at a time; bias,
//                   pre-activation, activation and residual in fp32, one rounding, through shared
//                   memory to TMA stores (or, for outputs TMA cannot address, to stores of 64
//                   consecutive bytes per row). Four warps per scheduler
//                   hide one another's waits: with two, a tile's epilogue took 11 us against 20 us
//                   of MMAs at K = 4096 (bias, GELU, residual and pre-activation).
// Either operand may be stored with k or with its other dimension contiguous: TMA boxes and the
// MMA descriptors differ, the arithmetic does not, so the three products of a linear layer and
// its gradient need no transposed copies.
//
// Measured: 16384 x 14336 x 4096 bf16 with bias, GELU and kept pre-activation 1.10 ms (1,745 TFLOP/s;
// 1.27 ms when run without a pause, at the clocks that the power limit then leaves): bound by the
// tensor cores. 512 x 12288 x 4096: 48.5 us, two rounds of tiles for 1.26 (tensor pipe busy 63%).
// 4095 x 3001 x 1537 f16 with every epilogue part in unaligned rows: 56 us without the repacking, bound
// by the epilogue's 2-byte stores. (Asking L2 for operands 6 to 12 k-blocks ahead: 4 to 25% longer.)
//
// Every wait is bounded (ptx.cuh); a wait that expires ends the role, and the CTAs still meet at
// the final cluster barrier and free their TMEM.
#include "activation16.cuh"
#include "layer16.cuh"
#include "pair_gemm16.cuh"
#include "raster.cuh"
#include "stream16.cuh"

#include <algorithm>
#include <mutex>

namespace sg {
namespace {

constexpr int kBM = 128;  // rows per CTA (256 per pair)
constexpr int kBK = 64;   // k values per 128-byte swizzled row

constexpr int kBN = 256;
constexpr int kEpiWarps = 16;  // 4 row quarters x 4 groups of 64 columns
constexpr int kThreads = 128 + 32 * kEpiWarps;
constexpr uint32_t kPartBytes = kBM * kBK * 2;  // A's or B's share of a stage
constexpr uint32_t kStageBytes = 2 * kPartBytes;
constexpr int kStages = 6;
constexpr uint32_t kStoreBytes = 2048;  // 32 rows x 32 values
constexpr size_t kSmem = kStages * kStageBytes + kEpiWarps * kStoreBytes + (2 * kStages + 4) * 8 + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "ring and store buffers fit in shared memory");

struct PairProduct {
    int M, N, KB;  // KB: k-blocks
    int tiles_m, tiles_n, split, items;  // items: tiles x split pieces along k
    int piece0, tile0;                   // first piece and first counted tile in scratch (split > 1)
    int a_mn, b_mn;
    uint32_t idesc;
    uint16_t *D;
    long long ldd;
    int d_tma;  // the output's rows are addressable by TMA
};
struct PairParams {
    PairProduct g[kMaxProducts];
    int total_items;
    float *pieces;           // [pieces][2 CTAs][256 columns][128 rows]
    unsigned int *counters;  // [tiles][2 CTAs][epilogue warps], zero between calls
    // The epilogue's matrices, of a launch with one product.
    const uint16_t *bias;
    int act;
    const uint16_t *res;
    long long ldr;
    int res_vec;  // the residual's rows allow 16-byte loads of 8 values each
    uint16_t *pre;
    long long ldz;
    int z_tma;
};
struct PairMaps {
    CUtensorMap a[kMaxProducts], b[kMaxProducts], d[kMaxProducts], z;
};
constexpr int kGroupM = 8;  // tile rows of the raster's groups

// Item t of the launch: its product, tile and k-blocks [kb0, kb0 + n).
struct Item {
    int product, tile, piece, tm, tn, kb0, n;
    __device__ __forceinline__ Item(const PairParams &p, int t) {
        product = t >= p.g[0].items ? 1 : 0;
        const PairProduct &g = p.g[product];
        if (product) t -= p.g[0].items;
        tile = t / g.split;
        piece = t - tile * g.split;
        tile_coords(tile, g.tiles_m, g.tiles_n, kGroupM, tm, tn);
        kb0 = static_cast<int>(static_cast<long long>(piece) * g.KB / g.split);
        n = static_cast<int>((piece + 1LL) * g.KB / g.split) - kb0;
    }
};

// Calls body with the operands' layouts as compile-time constants.
template <typename Body>
__device__ __forceinline__ void with_layout(const PairProduct &g, Body body) {
    if (g.a_mn)
        body(std::true_type(), std::true_type());
    else if (g.b_mn)
        body(std::false_type(), std::true_type());
    else
        body(std::false_type(), std::false_type());
}

// A wait whose arrivals may come from the other CTA of the pair.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t *bar, uint32_t parity) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((spin & 63u) == 0u && globaltimer_ns() - t0 > kWaitLimitNs) {
            raise_fault(kFaultTimeout);
            return false;
        }
    }
}

// 16-byte chunk c (0..3) of row r (0..31) of a warp's 32 x 32 buffer: the 64-byte TMA
// swizzle, with which eight lanes' 16-byte accesses touch all banks once.
__device__ __forceinline__ uint32_t store_chunk(int r, int c) {
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void activate32(float (&v)[32], int act) {
    with_activation(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = activate16<decltype(a)::value>(v[i]);
    });
}

// One warp's 32 x 32 block of an output at (row0, col0): v is lane r's row. It goes through `buf`
// (which no earlier copy still reads) to a TMA store or, for rows TMA cannot address, to stores of
// one row per instruction. (Stores of 16 bytes per lane from the same buffer, in place of the TMA
// stores, cost 3 to 6% on the large products; 4-byte stores of two rows per instruction, in place
// of 2-byte ones of one row, 40% on the ragged one.)
template <typename T>
__device__ __forceinline__ void store_block(const float (&v)[32], uint8_t *buf, const CUtensorMap *map,
                                            int tma, uint16_t *out, long long ld, int M, int N, int row0,
                                            int col0, int lane) {
    using H = Half16<T>;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        uint4 q;
        q.x = H::narrow2(v[8 * c], v[8 * c + 1]);
        q.y = H::narrow2(v[8 * c + 2], v[8 * c + 3]);
        q.z = H::narrow2(v[8 * c + 4], v[8 * c + 5]);
        q.w = H::narrow2(v[8 * c + 6], v[8 * c + 7]);
        *reinterpret_cast<uint4 *>(buf + store_chunk(lane, c)) = q;
    }
    if (tma) {
        async_proxy_fence();
        __syncwarp();
        if (lane == 0) {
            tma_store_2d(map, buf, col0, row0);
            bulk_commit();
        }
        return;
    }
    __syncwarp();
    const int rows = min(32, M - row0);
    if (col0 + lane < N) {
        uint16_t *p = out + static_cast<long long>(row0) * ld + col0 + lane;
#pragma unroll 8
        for (int r = 0; r < rows; ++r)
            p[r * ld] = *reinterpret_cast<const uint16_t *>(buf + store_chunk(r, lane >> 3) + (lane & 7) * 2);
    }
    __syncwarp();
}

// The residual of a 32 x 32 block is fetched ahead of the arithmetic before it, four lanes to a row
// (whole 32-byte sectors, eight rows per instruction), and turned around through `buf` so that
// each lane gets its own row. Rows without 16-byte alignment are read as the aligned 4-byte words
// around them. raw[5 i ..]: row 8 i + lane / 4, values 8 (lane % 4) .. + 7.
__device__ __forceinline__ void fetch_residual(uint32_t (&raw)[20], const PairParams &p, int row0,
                                               int col0, int lane) {
    const int col = col0 + (lane & 3) * 8, count = min(8, p.g[0].N - col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = row0 + 8 * i + (lane >> 2);
        if (row >= p.g[0].M || count <= 0) continue;
        const uint16_t *src = p.res + static_cast<long long>(row) * p.ldr + col;
        if (p.res_vec) {
            const uint4 q = *reinterpret_cast<const uint4 *>(src);
            raw[5 * i] = q.x;
            raw[5 * i + 1] = q.y;
            raw[5 * i + 2] = q.z;
            raw[5 * i + 3] = q.w;
        } else {
            const uintptr_t a = reinterpret_cast<uintptr_t>(src);
            const uint32_t *w = reinterpret_cast<const uint32_t *>(a & ~static_cast<uintptr_t>(3));
            const int shift = static_cast<int>(a & 2u) >> 1;  // only words with a value of the row
#pragma unroll
            for (int k = 0; k < 5; ++k)
                if (2 * k - shift < count) raw[5 * i + k] = w[k];
        }
    }
}
template <typename T>
__device__ __forceinline__ void add_residual(float (&v)[32], uint32_t (&raw)[20], uint8_t *buf,
                                             const PairParams &p, int row0, int col0, int lane) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = 8 * i + (lane >> 2);
        if (!p.res_vec) {
            const uint16_t *src = p.res + static_cast<long long>(row0 + r) * p.ldr + col0;
            if (reinterpret_cast<uintptr_t>(src) & 2u) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    raw[5 * i + k] = __funnelshift_r(raw[5 * i + k], raw[5 * i + k + 1], 16);
            }
        }
        *reinterpret_cast<uint4 *>(buf + store_chunk(r, lane & 3)) =
            make_uint4(raw[5 * i], raw[5 * i + 1], raw[5 * i + 2], raw[5 * i + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 q = *reinterpret_cast<const uint4 *>(buf + store_chunk(lane, c));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const float2 f = Half16<T>::widen2(w[k]);
            v[8 * c + 2 * k] += f.x;
            v[8 * c + 2 * k + 1] += f.y;
        }
    }
    __syncwarp();
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    pair_gemm16_kernel(const __grid_constant__ PairMaps maps, const __grid_constant__ PairParams p) {
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    uint8_t *store_bufs = smem + kStages * kStageBytes;
    uint64_t *full = reinterpret_cast<uint64_t *>(store_bufs + kEpiWarps * kStoreBytes);
    uint64_t *empty = full + kStages;
    uint64_t *acc_full = empty + kStages;  // [2]
    uint64_t *acc_free = acc_full + 2;     // [2], the leader's are used
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&maps.a[0]);
        tma_prefetch_desc(&maps.b[0]);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&acc_full[j], 1);
            mbar_init(&acc_free[j], 2 * kEpiWarps);
        }
        mbar_init_fence();
    }
    if (warp == 2) tmem_alloc<2>(tmem_slot, 2 * kBN);
    tc_before_sync();
    cluster_sync();  // the pair's barriers exist before either CTA's copies complete on them
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    grid_dependents();  // after the TMEM allocation: a later kernel's CTA cannot take it first
    grid_dependency();

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = pair; t < p.total_items && ok; t += pairs) {
                const Item item(p, t);
                const CUtensorMap *ma = &maps.a[item.product], *mb = &maps.b[item.product];
                const int m0 = item.tm * 256 + static_cast<int>(rank) * kBM;
                const int n0 = item.tn * kBN + static_cast<int>(rank) * (kBN / 2);
                auto blocks = [&](auto a_layout, auto b_layout) {
                    constexpr bool a_mn = decltype(a_layout)::value, b_mn = decltype(b_layout)::value;
                    for (int kb = item.kb0; kb < item.kb0 + item.n; ++kb, ++it) {
                        const int s = it % kStages, k0 = kb * kBK;
                        if (it >= kStages && !mbar_wait_cluster(&empty[s], ((it / kStages) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        uint8_t *sa = smem + s * kStageBytes, *sb = sa + kPartBytes;
                        if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kStageBytes);
                        const uint32_t bar = map_to_rank(&full[s], 0);
                        if (a_mn) {
                            tma_load_2d_pair(sa, ma, bar, m0, k0);
                            tma_load_2d_pair(sa + 8192, ma, bar, m0 + 64, k0);
                        } else {
                            tma_load_2d_pair(sa, ma, bar, k0, m0);
                        }
                        if (b_mn) {
                            tma_load_2d_pair(sb, mb, bar, n0, k0);
                            tma_load_2d_pair(sb + 8192, mb, bar, n0 + 64, k0);
                        } else {
                            tma_load_2d_pair(sb, mb, bar, k0, n0);
                        }
                    }
                };
                with_layout(p.g[item.product], blocks);
            }
            // Shared memory must outlive every copy: the leader waits (bounded) for the last
            // stages of both CTAs; the final cluster barrier holds the other CTA until then.
            if (rank == 0)
                for (int j = it > kStages ? it - kStages : 0; j < it; ++j)
                    if (!mbar_wait_cluster(&full[j % kStages], (j / kStages) & 1)) break;
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int it = 0, j = 0;
            bool ok = true;
            for (int t = pair; t < p.total_items && ok; t += pairs, ++j) {
                const Item item(p, t);
                const int i = item.product;
                const int set = j & 1;
                if (j >= 2 && !mbar_wait_cluster(&acc_free[set], ((j >> 1) - 1) & 1)) break;
                tc_after_sync();
                const uint32_t d = tmem + static_cast<uint32_t>(set * kBN);
                const int KB = item.n;
                const uint32_t idesc = p.g[i].idesc;
                auto blocks = [&](auto a_layout, auto b_layout) {
                    constexpr bool a_mn = decltype(a_layout)::value, b_mn = decltype(b_layout)::value;
                    for (int kb = 0; kb < KB; ++kb, ++it) {
                        const int s = it % kStages;
                        if (!mbar_wait_cluster(&full[s], (it / kStages) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_after_sync();
                        const uint32_t sa = smem_addr(smem + s * kStageBytes), sb = sa + kPartBytes;
                        const uint64_t da = a_mn ? desc_mn_major(sa, 8192) : desc_k_major(sa);
                        const uint64_t db = b_mn ? desc_mn_major(sb, 8192) : desc_k_major(sb);
#pragma unroll
                        for (int k = 0; k < kBK / 16; ++k)  // start addresses count 16 bytes: a
                            mma_16<2>(d, da + static_cast<uint64_t>(k * (a_mn ? 128 : 2)),  // k-step is
                                      db + static_cast<uint64_t>(k * (b_mn ? 128 : 2)),     // 32 bytes
                                      idesc, kb > 0 || k > 0);  // of a row or 16 rows
                        mma_commit_16<2>(&empty[s]);
                    }
                };
                with_layout(p.g[i], blocks);
                if (ok) mma_commit_16<2>(&acc_full[set]);
            }
        }
    } else if (warp >= 4) {
        const int w = warp - 4, quarter = warp & 3, group = w >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t *buf = store_bufs + w * kStoreBytes;
        const uint32_t free0 = map_to_rank(&acc_free[0], 0), free1 = map_to_rank(&acc_free[1], 0);
        const int c0 = group * 64;
        int j = 0;
        uint32_t raw[20];  // the next block's residual
        float bias[2] = {0.0f, 0.0f};  // of columns col0 + lane and col0 + 32 + lane
        for (int t = pair; t < p.total_items; t += pairs, ++j) {
            const int set = j & 1;
            const Item item(p, t);
            const PairProduct g = p.g[item.product];
            const int row0 = item.tm * 256 + static_cast<int>(rank) * kBM + quarter * 32;
            const int col0 = item.tn * kBN + c0;
            const bool inside = row0 < g.M && col0 < g.N;
            const int blocks = g.N - col0 > 32 ? 2 : 1;
            if (inside && g.split == 1) {
                if (p.res) fetch_residual(raw, p, row0, col0, lane);
                if (p.bias) {
                    bias[0] = col0 + lane < g.N ? Half16<T>::widen(p.bias[col0 + lane]) : 0.0f;
                    bias[1] = g.N - col0 - 32 > lane ? Half16<T>::widen(p.bias[col0 + 32 + lane]) : 0.0f;
                }
            }
            if (!mbar_wait_cluster(&acc_full[set], (j >> 1) & 1)) break;
            tc_after_sync();
            const uint32_t tset = tmem + lane_base + static_cast<uint32_t>(set * kBN + c0);
            auto release = [&]() {  // the warp's last read of this accumulator
                tc_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_at(set ? free1 : free0);
            };
            if (!inside) {
                release();
                continue;
            }
            const float *pieces = nullptr;  // of this lane's row, the tile's first one
            constexpr size_t kPiece = 2ull * kBN * kBM;
            if (g.split > 1) {
                const size_t at = static_cast<size_t>(g.piece0 + item.tile * g.split);
                float *base = p.pieces + (2 * at + rank) * kBN * kBM + c0 * kBM + quarter * 32 + lane;
#pragma unroll 1
                for (int b = 0; b < 2; ++b) {
                    uint32_t r[32];
                    tmem_ld_x32(tset + static_cast<uint32_t>(32 * b), r);
                    tmem_ld_wait();
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        __stcg(base + item.piece * kPiece + (32 * b + i) * kBM, __uint_as_float(r[i]));
                }
                release();
                unsigned int *counter =
                    p.counters + (2 * static_cast<size_t>(g.tile0 + item.tile) + rank) * kEpiWarps + w;
                if (!piece_arrived(counter, 1, g.split, lane)) continue;
                pieces = base;
                if (p.res) fetch_residual(raw, p, row0, col0, lane);
                if (p.bias) {
                    bias[0] = col0 + lane < g.N ? Half16<T>::widen(p.bias[col0 + lane]) : 0.0f;
                    bias[1] = g.N - col0 - 32 > lane ? Half16<T>::widen(p.bias[col0 + 32 + lane]) : 0.0f;
                }
            }
            // The product's 32 columns of block b: the accumulator, or the pieces in the order of k.
            auto values = [&](int b, float(&v)[32]) {
                if (pieces) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = 0.0f;
                    for (int k = 0; k < g.split; ++k)
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] += __ldcg(pieces + k * kPiece + (32 * b + i) * kBM);
                } else {
                    tmem_ld_x32(tset + static_cast<uint32_t>(32 * b), reinterpret_cast<uint32_t(&)[32]>(v));
                    tmem_ld_wait();
                }
            };
#pragma unroll 1
            for (int b = 0; b < blocks; ++b) {
                const int col = col0 + 32 * b;
                float v[32];
                values(b, v);
                if (b == blocks - 1 && !pieces) release();
                if (p.bias) {
                    const float mine = b ? bias[1] : bias[0];
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, mine, i);
                }
                if (p.pre) {
                    if (lane == 0) bulk_wait_read<0>();
                    __syncwarp();
                    store_block<T>(v, buf, &maps.z, p.z_tma, p.pre, p.ldz, g.M, g.N, row0, col, lane);
                }
                activate32(v, p.act);
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
                if (p.res) {
                    add_residual<T>(v, raw, buf, p, row0, col, lane);
                    if (b + 1 < blocks) fetch_residual(raw, p, row0, col + 32, lane);
                }
                store_block<T>(v, buf, &maps.d[item.product], g.d_tma, g.D, g.ldd, g.M, g.N, row0, col, lane);
            }
        }
        if (lane == 0) bulk_wait_read<0>();
    }

    __syncwarp();
    tc_before_sync();
    cluster_sync();  // neither CTA's shared or tensor memory is used by the other any more
    if (warp == 2) {
        tc_after_sync();
        tmem_dealloc<2>(tmem, 2 * kBN);
    }
}

// ---- host side ------------------------------------------------------------------------------------

constexpr int kMaxDevices = 64;

// Pairs that can run at once (an odd SM of a cluster group stays idle), found once per device.
template <typename T>
cudaError_t prepare(int dev, int *pairs) {
    static std::once_flag once[kMaxDevices];
    static cudaError_t setup[kMaxDevices];
    static int max_pairs[kMaxDevices];
    std::call_once(once[dev], [&] {
        auto kernel = pair_gemm16_kernel<T>;
        setup[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(kSmem));
        if (setup[dev] != cudaSuccess) return;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2, 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = kSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        setup[dev] = cudaOccupancyMaxActiveClusters(&max_pairs[dev], kernel, &cfg);
        if (setup[dev] == cudaSuccess && max_pairs[dev] < 1) setup[dev] = cudaErrorInvalidConfiguration;
    });
    *pairs = max_pairs[dev];
    return setup[dev];
}

// Cuts the tiles of each product into up to 8 pieces along k where that shortens the launch. The pairs
// take the items in turn, so the busiest has a count that follows from the sizes; a k-block takes
// 0.31 us, a piece 0.085 us to write and read (256 KiB at 3 TB/s), and summing s of them 2 s us. (bf16:
// gradients of 6338 rows 80 -> 288, two tiles of 100 blocks for dW: 41 us whole, 28 cut. 512 x 4096 x
// 14336, 32 tiles of 224 blocks: 73 and 51. 512 x 12288 x 14336, 96 tiles: 147 and 130. 1024 x 4096 x
// 4096, 64 tiles of 64 blocks, stays whole: 27, 40 cut in two.) A product's items are four rounds of the
// pairs at most, its pieces 80 MB.
void cut_along_k(PairParams &p, int n, int pairs) {
    PairProduct &a = p.g[0], &b = p.g[1];
    const int tiles_a = a.items, tiles_b = n == 2 ? b.items : 0, kb_b = n == 2 ? b.KB : 1;
    double best = 0.0;
    auto most = [&](int tiles, int kb) {
        return tiles == 0 ? 1 : std::max(1, std::min({8, kb, 4 * pairs / tiles}));
    };
    for (int sa = 1; sa <= most(tiles_a, a.KB); ++sa) {
        for (int sb = 1; sb <= most(tiles_b, kb_b); ++sb) {
            // The first product's items come first; the second's go on where they end.
            const int na = tiles_a * sa, nb = tiles_b * sb, ra = na % pairs, rb = nb % pairs;
            const double ka = (a.KB + sa - 1) / sa, kb = (kb_b + sb - 1) / sb;
            const double one = ra ? (na / pairs + 1) * ka + (nb / pairs + (ra + rb > pairs)) * kb : 0.0;
            const double two = (na / pairs) * ka + (nb / pairs + (rb > 0)) * kb;
            const double us = 0.31 * std::max(one, two) + 0.085 * ((sa > 1 ? na : 0) + (sb > 1 ? nb : 0)) +
                              (sa > 1 || sb > 1 ? 2.0 * std::max(sa, sb) : 0.0);
            if (best == 0.0 || us < best) {
                best = us;
                a.split = sa;
                a.items = na;
                if (n == 2) {
                    b.split = sb;
                    b.items = nb;
                }
            }
        }
    }
}

template <typename T>
cudaError_t launch(const Gemm16 *list, int n, cudaStream_t stream, const char **detail) {
    int dev = 0, max_pairs = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        *detail = "cudaGetDevice failed";
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    }
    err = prepare<T>(dev, &max_pairs);
    if (err != cudaSuccess) {
        *detail = "linear layer kernel set-up failed";
        return err;
    }
    PairParams p = {};
    PairMaps maps;
    // Tiles with the longer k first: the shorter ones fill the last round.
    const int order[2] = {n == 2 && list[1].K > list[0].K ? 1 : 0, n == 2 && list[1].K > list[0].K ? 0 : 1};
    for (int i = 0; i < n; ++i) {
        const Gemm16 &g = list[order[i]];
        PairProduct &q = p.g[i];
        q.M = g.M;
        q.N = g.N;
        q.KB = static_cast<int>((g.K + static_cast<long long>(kBK) - 1) / kBK);
        q.tiles_m = static_cast<int>((g.M + 255LL) / 256);
        q.tiles_n = static_cast<int>((g.N + static_cast<long long>(kBN) - 1) / kBN);
        const long long tiles = static_cast<long long>(q.tiles_m) * q.tiles_n;
        if (tiles > 0x3fffffffLL) {
            *detail = "too many output tiles";
            return cudaErrorInvalidValue;
        }
        q.split = 1;
        q.items = static_cast<int>(tiles);
        q.a_mn = g.a_mn;
        q.b_mn = g.b_mn;
        q.idesc = idesc_16(256, kBN, Half16<T>::kind, g.a_mn, g.b_mn);
        q.D = g.D;
        q.ldd = g.ldd;
        // A TMA store also writes zeros into the rest of a row's last 16 bytes, which may belong to
        // the caller's wider matrix: only rows that end on that boundary are stored so.
        q.d_tma = tma_rows(g.D, g.ldd) && g.N % 8 == 0;
        if (!(g.a_mn ? tensor_map_16(&maps.a[i], g.A, g.dtype, g.M, g.K, g.lda, 64, kBK)
                     : tensor_map_16(&maps.a[i], g.A, g.dtype, g.K, g.M, g.lda, kBK, kBM)) ||
            !(g.b_mn ? tensor_map_16(&maps.b[i], g.B, g.dtype, g.N, g.K, g.ldb, 64, kBK)
                     : tensor_map_16(&maps.b[i], g.B, g.dtype, g.K, g.N, g.ldb, kBK, kBN / 2)) ||
            (q.d_tma && !tensor_map_16(&maps.d[i], g.D, g.dtype, g.N, g.M, g.ldd, 32, 32, true))) {
            *detail = "cuTensorMapEncodeTiled rejected a matrix";
            return cudaErrorInvalidValue;
        }
    }
    cut_along_k(p, n, max_pairs);
    size_t pieces = 0, cut_tiles = 0;
    for (int i = 0; i < n; ++i) {
        PairProduct &q = p.g[i];
        if (q.split > 1) {
            q.piece0 = static_cast<int>(pieces);
            q.tile0 = static_cast<int>(cut_tiles);
            pieces += static_cast<size_t>(q.items);
            cut_tiles += static_cast<size_t>(q.items / q.split);
        }
        p.total_items += q.items;
    }
    if (pieces > 0) {
        void *data = nullptr, *sync = nullptr;
        err = layer_scratch(kScratchPair, stream, pieces * 2 * kBN * kBM * 4, &data, detail);
        if (err == cudaSuccess)
            err = layer_scratch(kScratchPairSync, stream, cut_tiles * 2 * kEpiWarps * 4, &sync, detail);
        if (err != cudaSuccess) return err;
        p.pieces = static_cast<float *>(data);
        p.counters = static_cast<unsigned int *>(sync);
    }
    if (n == 1) {
        const Gemm16 &g = list[0];
        p.bias = g.bias;
        p.act = g.act;
        p.res = g.res;
        p.ldr = g.ldr;
        p.res_vec = g.res && tma_rows(g.res, g.ldr) && g.N % 8 == 0;
        p.pre = g.pre;
        p.ldz = g.ldz;
        p.z_tma = g.pre && tma_rows(g.pre, g.ldz) && g.N % 8 == 0;
        if (p.z_tma && !tensor_map_16(&maps.z, g.pre, g.dtype, g.N, g.M, g.ldz, 32, 32, true)) {
            *detail = "cuTensorMapEncodeTiled rejected a matrix";
            return cudaErrorInvalidValue;
        }
    }
    const int pairs = std::min(p.total_items, max_pairs);
    err = launch_early(pair_gemm16_kernel<T>, dim3(2u * static_cast<unsigned>(pairs)), kThreads, kSmem,
                       stream, maps, p);
    if (err != cudaSuccess) *detail = "linear layer kernel launch failed";
    return err;
}

}  // namespace

cudaError_t pair_gemm16_launch(const Gemm16 *list, int n, cudaStream_t stream, const char **detail) {
    return list[0].dtype == kBf16 ? launch<__nv_bfloat16>(list, n, stream, detail)
                                  : launch<__half>(list, n, stream, detail);
}

// ---- tensor maps ------------------------------------------------------------------------------------

namespace {
using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                   const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                   const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_fn() {
    static const EncodeTiledFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                             cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeTiledFn>(f);
    }();
    return fn;
}
}  // namespace

bool tensor_map_16(CUtensorMap *map, const void *base, int dtype, long long cols, long long rows,
                   long long ld, int box_cols, int box_rows, bool narrow, long long depth,
                   long long stride) {
    const EncodeTiledFn enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows),
                                static_cast<cuuint64_t>(depth)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld) * 2, static_cast<cuuint64_t>(stride) * 2};
    const cuuint32_t box[3] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1};
    const cuuint32_t estr[3] = {1, 1, 1};
    return enc(map, dtype == kBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
               depth > 0 ? 3 : 2, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               narrow ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sg
