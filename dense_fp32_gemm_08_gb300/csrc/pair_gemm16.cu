// pair_gemm16.cu: D = act(A . B + bias) + res on 16-bit values with tcgen05 MMAs over pairs of
// CTAs (cta_group::2): one MMA multiplies 256 rows by BN columns, each CTA of the pair holding
// half of A's rows and half of B's columns in its own shared memory, so each SM stages half the
// operand bytes per multiply-add of a one-CTA tile.
//
// A persistent grid of pairs walks the 256 x BN output tiles in grouped-raster order. Roles of a
// CTA's 12 warps:
//   warp 0, lane 0: TMA producer: this CTA's 128 rows of A and BN / 2 columns of B per 64-wide
//                   k-block into a ring of STAGES stages; both CTAs' copies complete on the
//                   leader's "full" barrier.
//   warp 1, lane 0: (leader CTA) issues the MMAs, four k-steps of 16 per block, into one of two
//                   TMEM accumulators of BN columns; commits free the stage in both CTAs and,
//                   at a tile's end, hand the accumulator to both CTAs' epilogues.
//   warp 2:         allocates and frees the pair's TMEM.
//   warps 4..11:    epilogue of this CTA's 128 rows while the next tile multiplies: warp w reads
//                   TMEM lanes 32 (w % 4) .. + 31 and one half of the columns, 32 at a time;
//                   bias, pre-activation, activation and residual in fp32, one rounding, through
//                   shared memory to TMA stores (or, for outputs TMA cannot address, to stores
//                   of 64 consecutive bytes per row).
// Either operand may be stored with k or with its other dimension contiguous: TMA boxes and the
// MMA descriptors differ, the arithmetic does not, so the three products of a linear layer and
// its gradient need no transposed copies.
//
// Every wait is bounded (ptx.cuh); a wait that expires ends the role, and the CTAs still meet at
// the final cluster barrier and free their TMEM.
#include "activation16.cuh"
#include "layer16.cuh"
#include "pair_gemm16.cuh"
#include "raster.cuh"
#include "tc16.cuh"

#include <algorithm>
#include <mutex>

namespace sg {
namespace {

constexpr int kBM = 128;  // rows per CTA (256 per pair)
constexpr int kBK = 64;   // k values per 128-byte swizzled row
constexpr int kEpiWarps = 8;
constexpr int kThreads = 128 + 32 * kEpiWarps;

struct PairParams {
    int M, N, K;
    int tiles_m, tiles_n, group_m, total_tiles;
    uint32_t idesc;
    const uint16_t *bias;
    int act;
    const uint16_t *res;
    long long ldr;
    uint16_t *D;
    long long ldd;
    uint16_t *pre;
    long long ldz;
    int d_tma, z_tma;  // the output's rows are addressable by TMA
    int res_vec;       // the residual's rows allow 16-byte loads
};

template <int BN>
struct PairConfig {
    static constexpr uint32_t A_BYTES = kBM * kBK * 2;
    static constexpr uint32_t B_BYTES = (BN / 2) * kBK * 2;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int STAGES = BN == 256 ? 6 : 8;
    static constexpr uint32_t STORE_BYTES = 2048;  // 32 rows x 32 values
    static constexpr uint32_t TMEM_COLS = 2 * BN;
    static constexpr size_t SMEM = STAGES * STAGE_BYTES + kEpiWarps * 2 * STORE_BYTES +
                                   (2 * STAGES + 4) * 8 + 16 + 1024;
};

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

// 16-byte chunk c (0..3) of row r (0..31) of a warp's 32 x 32 store tile: the 64-byte TMA swizzle,
// with which eight lanes' 16-byte accesses touch all banks once.
__device__ __forceinline__ uint32_t store_chunk(int r, int c) {
    return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

__device__ __forceinline__ void activate32(float (&v)[32], int act) {
    with_activation(act, [&](auto a) {
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = activate16<decltype(a)::value>(v[i]);
    });
}

// One warp's 32 x 32 block of an output at (row0, col0): v is lane r's row. `buf` is free (no
// copy reads it) on entry for every lane.
template <typename T>
__device__ __forceinline__ void store_block(const float (&v)[32], uint8_t *buf,
                                            const CUtensorMap *map, int tma, uint16_t *out,
                                            long long ld, int M, int N, int row0, int col0,
                                            int lane) {
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
    } else {
        __syncwarp();
        const int rows = min(32, M - row0);
        uint16_t *p = out + static_cast<long long>(row0) * ld + col0 + lane;
        if (col0 + lane < N) {
#pragma unroll 8
            for (int r = 0; r < rows; ++r)
                p[r * ld] = *reinterpret_cast<const uint16_t *>(buf + store_chunk(r, lane >> 3) + (lane & 7) * 2);
        }
        __syncwarp();
    }
}

// The residual's 32 values of lane r's row, added to v. Rows that allow it are read 16 bytes at a
// time by their own lane; otherwise the warp reads 64 consecutive bytes of one row after another
// and hands them over through `buf`.
template <typename T>
__device__ __forceinline__ void add_residual(float (&v)[32], uint8_t *buf, const PairParams &p,
                                             int row0, int col0, int lane) {
    using H = Half16<T>;
    if (p.res_vec && col0 + 32 <= p.N) {
        if (row0 + lane < p.M) {
            const uint4 *src = reinterpret_cast<const uint4 *>(
                p.res + static_cast<long long>(row0 + lane) * p.ldr + col0);
            uint4 q[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) q[c] = src[c];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const uint32_t w[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 f = H::widen2(w[i]);
                    v[8 * c + 2 * i] += f.x;
                    v[8 * c + 2 * i + 1] += f.y;
                }
            }
        }
        return;
    }
    const uint16_t *src = p.res + static_cast<long long>(row0) * p.ldr + col0 + lane;
    const int rows = min(32, p.M - row0);
    uint16_t t[32];
#pragma unroll
    for (int r = 0; r < 32; ++r) t[r] = r < rows && col0 + lane < p.N ? src[r * p.ldr] : uint16_t(0);
#pragma unroll
    for (int r = 0; r < 32; ++r)
        *reinterpret_cast<uint16_t *>(buf + store_chunk(r, lane >> 3) + (lane & 7) * 2) = t[r];
    __syncwarp();
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint4 q = *reinterpret_cast<const uint4 *>(buf + store_chunk(lane, c));
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = H::widen2(w[i]);
            v[8 * c + 2 * i] += f.x;
            v[8 * c + 2 * i + 1] += f.y;
        }
    }
    __syncwarp();
}

template <int BN, bool A_MN, bool B_MN, typename T>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
    pair_gemm16_kernel(const __grid_constant__ CUtensorMap map_a,
                       const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_d,
                       const __grid_constant__ CUtensorMap map_z, const PairParams p) {
    using C = PairConfig<BN>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    uint8_t *store_bufs = smem + STAGES * C::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(store_bufs + kEpiWarps * 2 * C::STORE_BYTES);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;  // [2]
    uint64_t *acc_free = acc_full + 2;    // [2], the leader's are used
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const int KB = (p.K + kBK - 1) / kBK;

    if (threadIdx.x == 0) {
        tma_prefetch_desc(&map_a);
        tma_prefetch_desc(&map_b);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&acc_full[j], 1);
            mbar_init(&acc_free[j], 2 * kEpiWarps);
        }
        mbar_init_fence();
    }
    if (warp == 2) tmem_alloc<2>(tmem_slot, C::TMEM_COLS);
    tc_before_sync();
    __syncthreads();
    cluster_sync();  // the pair's barriers exist before either CTA's copies complete on them
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        if (lane == 0) {
            int it = 0;
            bool ok = true;
            for (int t = pair; t < p.total_tiles && ok; t += pairs) {
                int tm, tn;
                tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
                const int m0 = tm * 256 + static_cast<int>(rank) * kBM;
                const int n0 = tn * BN + static_cast<int>(rank) * (BN / 2);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (it >= STAGES && !mbar_wait_cluster(&empty[s], ((it / STAGES) - 1) & 1)) {
                        ok = false;
                        break;
                    }
                    uint8_t *sa = smem + s * C::STAGE_BYTES, *sb = sa + C::A_BYTES;
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * C::STAGE_BYTES);
                    const uint32_t bar = map_to_rank(&full[s], 0);
                    const int k0 = kb * kBK;
                    if (A_MN) {
#pragma unroll
                        for (int i = 0; i < kBM / 64; ++i)
                            tma_load_2d_pair(sa + i * 8192, &map_a, bar, m0 + 64 * i, k0);
                    } else {
                        tma_load_2d_pair(sa, &map_a, bar, k0, m0);
                    }
                    if (B_MN) {
#pragma unroll
                        for (int i = 0; i < BN / 128; ++i)
                            tma_load_2d_pair(sb + i * 8192, &map_b, bar, n0 + 64 * i, k0);
                    } else {
                        tma_load_2d_pair(sb, &map_b, bar, k0, n0);
                    }
                }
            }
            // Shared memory must outlive every copy: the leader waits (bounded) for the last
            // stages of both CTAs; the final cluster barrier holds the other CTA until then.
            if (rank == 0)
                for (int j = it > STAGES ? it - STAGES : 0; j < it; ++j)
                    if (!mbar_wait_cluster(&full[j % STAGES], (j / STAGES) & 1)) break;
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            int it = 0, j = 0;
            bool ok = true;
            for (int t = pair; t < p.total_tiles && ok; t += pairs, ++j) {
                const int set = j & 1;
                if (j >= 2 && !mbar_wait_cluster(&acc_free[set], ((j >> 1) - 1) & 1)) break;
                tc_after_sync();
                const uint32_t d = tmem + static_cast<uint32_t>(set * BN);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % STAGES;
                    if (!mbar_wait_cluster(&full[s], (it / STAGES) & 1)) {
                        ok = false;
                        break;
                    }
                    tc_after_sync();
                    const uint32_t sa = smem_addr(smem + s * C::STAGE_BYTES), sb = sa + C::A_BYTES;
                    const uint64_t da = A_MN ? desc_mn_major(sa, 8192) : desc_k_major(sa);
                    const uint64_t db = B_MN ? desc_mn_major(sb, 8192) : desc_k_major(sb);
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)  // start addresses count 16 bytes
                        mma_16<2>(d, da + static_cast<uint64_t>(k * (A_MN ? 128 : 2)),
                                  db + static_cast<uint64_t>(k * (B_MN ? 128 : 2)), p.idesc,
                                  kb > 0 || k > 0);
                    mma_commit_16<2>(&empty[s]);
                }
                if (ok) mma_commit_16<2>(&acc_full[set]);
            }
        }
    } else if (warp >= 4) {
        const int w = warp - 4, quarter = warp & 3, half = w >> 2;
        const uint32_t lane_base = static_cast<uint32_t>(quarter * 32) << 16;
        uint8_t *bufs = store_bufs + w * 2 * C::STORE_BYTES;
        const uint32_t free0 = map_to_rank(&acc_free[0], 0), free1 = map_to_rank(&acc_free[1], 0);
        int j = 0, nbuf = 0;
        for (int t = pair; t < p.total_tiles; t += pairs, ++j) {
            const int set = j & 1;
            if (!mbar_wait_cluster(&acc_full[set], (j >> 1) & 1)) break;
            tc_after_sync();
            int tm, tn;
            tile_coords(t, p.tiles_m, p.tiles_n, p.group_m, tm, tn);
            const int row0 = tm * 256 + static_cast<int>(rank) * kBM + quarter * 32;
            const uint32_t tset = tmem + lane_base + static_cast<uint32_t>(set * BN);
#pragma unroll 1
            for (int c0 = half * (BN / 2); c0 < (half + 1) * (BN / 2); c0 += 32) {
                uint32_t r[32];
                tmem_ld_x32(tset + static_cast<uint32_t>(c0), r);
                tmem_ld_wait();
                if (c0 + 32 == (half + 1) * (BN / 2)) {  // the warp's last read of this accumulator
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_at(set ? free1 : free0);
                }
                const int col0 = tn * BN + c0;
                if (row0 >= p.M || col0 >= p.N) continue;
                float v[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
                if (p.bias) {
                    const float b = col0 + lane < p.N ? Half16<T>::widen(p.bias[col0 + lane]) : 0.0f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] += __shfl_sync(0xFFFFFFFFu, b, i);
                }
                if (p.pre) {
                    if (lane == 0) bulk_wait_read<1>();
                    __syncwarp();
                    store_block<T>(v, bufs + nbuf * C::STORE_BYTES, &map_z, p.z_tma, p.pre, p.ldz, p.M,
                                   p.N, row0, col0, lane);
                    nbuf ^= 1;
                }
                activate32(v, p.act);
                if (lane == 0) bulk_wait_read<1>();
                __syncwarp();
                if (p.res) add_residual<T>(v, bufs + nbuf * C::STORE_BYTES, p, row0, col0, lane);
                store_block<T>(v, bufs + nbuf * C::STORE_BYTES, &map_d, p.d_tma, p.D, p.ldd, p.M, p.N,
                               row0, col0, lane);
                nbuf ^= 1;
            }
        }
        if (lane == 0) bulk_wait<0>();
    }

    __syncwarp();
    tc_before_sync();
    __syncthreads();
    cluster_sync();  // neither CTA's shared or tensor memory is used by the other any more
    if (warp == 2) {
        tc_after_sync();
        tmem_dealloc<2>(tmem, C::TMEM_COLS);
    }
}

// ---- host side ------------------------------------------------------------------------------------

constexpr int kMaxDevices = 64;

template <int BN, bool A_MN, bool B_MN, typename T>
cudaError_t launch(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    using C = PairConfig<BN>;
    auto kernel = pair_gemm16_kernel<BN, A_MN, B_MN, T>;
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        *detail = "cudaGetDevice failed";
        return err != cudaSuccess ? err : cudaErrorInvalidDevice;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    // Pairs that can run at once (an odd SM of a cluster group stays idle), queried once.
    static std::once_flag once[kMaxDevices];
    static cudaError_t setup[kMaxDevices];
    static int max_pairs[kMaxDevices];
    std::call_once(once[dev], [&] {
        setup[dev] = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(C::SMEM));
        if (setup[dev] != cudaSuccess) return;
        cudaLaunchConfig_t q = cfg;
        q.gridDim = dim3(2, 1, 1);
        q.attrs = attr;
        q.numAttrs = 1;
        setup[dev] = cudaOccupancyMaxActiveClusters(&max_pairs[dev], kernel, &q);
        if (setup[dev] == cudaSuccess && max_pairs[dev] < 1) setup[dev] = cudaErrorInvalidConfiguration;
    });
    if (setup[dev] != cudaSuccess) {
        *detail = "linear layer kernel set-up failed";
        return setup[dev];
    }

    PairParams p;
    p.M = g.M;
    p.N = g.N;
    p.K = g.K;
    p.tiles_m = static_cast<int>((g.M + 255LL) / 256);
    p.tiles_n = static_cast<int>((g.N + static_cast<long long>(BN) - 1) / BN);
    p.group_m = 8;
    const long long tiles = static_cast<long long>(p.tiles_m) * p.tiles_n;
    if (tiles > 0x3fffffffLL) {
        *detail = "too many output tiles";
        return cudaErrorInvalidValue;
    }
    p.total_tiles = static_cast<int>(tiles);
    p.idesc = idesc_16(256, BN, Half16<T>::kind, A_MN, B_MN);
    p.bias = g.bias;
    p.act = g.act;
    p.res = g.res;
    p.ldr = g.ldr;
    p.D = g.D;
    p.ldd = g.ldd;
    p.pre = g.pre;
    p.ldz = g.ldz;
    // A TMA store also writes zeros into the rest of a row's last 16 bytes, which may belong to
    // the caller's wider matrix: only rows that end on that boundary are stored so.
    p.d_tma = tma_rows(g.D, g.ldd) && g.N % 8 == 0;
    p.z_tma = g.pre && tma_rows(g.pre, g.ldz) && g.N % 8 == 0;
    p.res_vec = g.res && tma_rows(g.res, g.ldr);

    CUtensorMap ma, mb, md, mz;
    const bool ok =
        (A_MN ? tensor_map_16(&ma, g.A, g.dtype, g.M, g.K, g.lda, 64, kBK, 128)
              : tensor_map_16(&ma, g.A, g.dtype, g.K, g.M, g.lda, kBK, kBM, 128)) &&
        (B_MN ? tensor_map_16(&mb, g.B, g.dtype, g.N, g.K, g.ldb, 64, kBK, 128)
              : tensor_map_16(&mb, g.B, g.dtype, g.K, g.N, g.ldb, kBK, BN / 2, 128)) &&
        (!p.d_tma || tensor_map_16(&md, g.D, g.dtype, g.N, g.M, g.ldd, 32, 32, 64)) &&
        (!p.z_tma || tensor_map_16(&mz, g.pre, g.dtype, g.N, g.M, g.ldz, 32, 32, 64));
    if (!ok) {
        *detail = "cuTensorMapEncodeTiled rejected a matrix";
        return cudaErrorInvalidValue;
    }
    if (!p.d_tma) md = ma;
    if (!p.z_tma) mz = ma;
    const int pairs = static_cast<int>(std::min<long long>(tiles, max_pairs[dev]));
    cfg.gridDim = dim3(2u * static_cast<unsigned>(pairs), 1, 1);
    err = cudaLaunchKernelEx(&cfg, kernel, ma, mb, md, mz, p);
    if (err == cudaSuccess) err = cudaGetLastError();
    if (err != cudaSuccess) *detail = "linear layer kernel launch failed";
    return err;
}

template <int BN, typename T>
cudaError_t launch_major(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    if (g.a_mn) return launch<BN, true, true, T>(g, stream, detail);
    return g.b_mn ? launch<BN, false, true, T>(g, stream, detail)
                  : launch<BN, false, false, T>(g, stream, detail);
}

}  // namespace

cudaError_t pair_gemm16_launch(const Gemm16 &g, cudaStream_t stream, const char **detail) {
    return g.dtype == kBf16 ? launch_major<256, __nv_bfloat16>(g, stream, detail)
                            : launch_major<256, __half>(g, stream, detail);
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
                   long long ld, int box_cols, int box_rows, int swizzle_bytes, long long depth,
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
               swizzle_bytes == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace sg
