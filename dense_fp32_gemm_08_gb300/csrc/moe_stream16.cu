// moe_stream16.cu: a whole mixture-of-experts layer for a few tokens in one kernel.
//
// The layer is bound by reading the chosen experts' weights once: 2 bytes per weight against
// 2 x (tokens of that expert) operations. One cooperative grid, one CTA per SM, runs four steps
// with a grid barrier between them, so that nothing but the weights moves far:
//   1. scores s = X . Wr^T, an expert and 8 tokens per CTA in turn, fp32 FMAs (every CTA for itself,
//      without the barrier, for up to 8 scores);
//   2. routing, computed by every CTA for itself (a few hundred values): softmax statistics in
//      fp32, the k largest scores with ties to the lowest index, and the list of chosen experts
//      with their tokens as 64-bit masks;
//   3. h = act(gate) * up: weights stream through a TMA ring into tcgen05 MMAs (stream16.cuh)
//      against all tokens; the epilogue keeps the columns of the expert's own tokens;
//   4. the experts' outputs, the same way against the rows of h; then every output value sums
//      its token's experts in the order of their rank, adds the residual and is rounded once.
// The ring runs across the barrier between 3 and 4: the weights of step 4 do not depend on h, so
// the first stages are under way before h is complete.
//
// Measured, one token through 2 of 8 experts of 4096 x 14336 bf16 (704 MB of weights): 131 us, 5.4
// TB/s: scores and routing 4.4, step 3 77 (6.1 TB/s), its barrier 6, step 4 38 (6.2 TB/s), its barrier
// 2.8, the sum 1. 24 tokens through 64 experts of 2048 x 1024 f16 (774 MB): 164 us, 4.7 TB/s; DRAM reads
// 777 MB. The memory's rate bounds the steps, the slowest CTA's pieces the barriers. (Sending the next
// weights to L2 during the barrier or the routing, 10 to 64 blocks per CTA, made it 1 to 5% slower.)
//
// h is rounded to the call's 16-bit type, as the tensor cores need it and as a layer computed in
// separate products would hold it; every sum is in fp32, cut tiles are summed in the order of k.
// A row of h with a finite value past half's 65,504 is held divided by a power of two: step 3 keeps
// the values that do not fit, and the row's largest, in fp32; after its barrier, and only in a call
// that has such a row, the epilogue's warps divide the row, a further barrier follows, and the
// sum at the end multiplies the expert's output by the same power. (24 tokens through 64 experts in
// half, no such row: 164.2 us; 163.9 without the check.)
#include "activation16.cuh"
#include "layer16.cuh"
#include "moe16.cuh"
#include "pair_gemm16.cuh"
#include "stream16.cuh"

#include <algorithm>
#include <mutex>

namespace sg {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kPairs = kMoeMaxTokens * kMoeMaxTopk;

// Grid barrier state, zero between calls (`gen` only counts up).
struct alignas(8) MoeSync {
    unsigned int count[4];
    unsigned int gen;
    unsigned int wide;  // half: set when a value of h is past the type's range; read with `gen`
    unsigned int done;  // CTAs at the end of such a call
    unsigned int largest[kPairs];  // the largest of a row's finite values past the range (as bits)
};
constexpr size_t kSyncBytes = (sizeof(MoeSync) + 255) / 256 * 256;

struct MoeParams {
    Moe16 m;
    int tiles_f, kb_up;    // step 3: tiles of one expert's F, k-blocks of D
    int tiles_d, kb_down;  // step 4: tiles of D, k-blocks of F
    uint32_t idesc;
    MoeSync *sync;
    unsigned int *counters;  // [active experts * tiles_f][epilogue warps]: units of step 3 that arrived
    float *score;            // [T][E]
    uint16_t *h;             // [T * k][ldh]
    long long ldh;
    float *wide;             // half: [T * k][F], values of h past the type's range
    float *out;              // [T * k][tiles_d * 128]: an expert's output for one token
    float *up_pieces;        // [2 * CTAs][accumulators][NT / 4][128][4]
    float *down_pieces;      // [2 * CTAs][NT][128]
};

// What every CTA knows of the routing.
struct Routing {
    unsigned long long mask[kMoeMaxExperts];  // tokens of an expert
    float weight[kPairs];
    uint16_t expert[kPairs];  // of (token, rank); kNone for an idle token
    uint16_t offset[kMoeMaxExperts];  // first row of h of an expert
    uint16_t rank[kMoeMaxExperts];    // position in `active`
    uint16_t active[kMoeMaxExperts];
    int n_active;
};
constexpr uint16_t kNone = 0xFFFF;

template <int NT, bool GATED>
struct MoeConfig {
    static constexpr int ACCS = GATED ? 2 : 1;
    static constexpr int GROUPS = NT / 32 > 0 ? NT / 32 : 1;  // of epilogue warps, 32 columns each
    static constexpr int THREADS = 128 + 128 * GROUPS;
    static constexpr uint32_t W_BYTES = kStreamRows * kStreamK * 2;
    static constexpr uint32_t A_BYTES = ACCS * W_BYTES;
    static constexpr uint32_t X_BYTES = NT * kStreamK * 2;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + X_BYTES;
    static constexpr size_t FIXED = sizeof(Routing) + 1024 + 512;
    static constexpr int FIT = static_cast<int>((227 * 1024 - FIXED) / STAGE_BYTES);
    static constexpr int STAGES = FIT < 11 ? FIT : 11;
    static constexpr uint32_t TMEM_COLS = 2 * ACCS * NT < 32 ? 32 : 2 * ACCS * NT;
    static constexpr size_t SMEM = STAGES * STAGE_BYTES + FIXED;
};

__device__ __forceinline__ void grid_arrive(unsigned int *count, unsigned int *gen, unsigned int ctas) {
    __threadfence();
    if (atomicAdd(count, 1u) == ctas - 1) {
        atomicExch(count, 0u);
        __threadfence();
        atomicAdd(gen, 1u);
    }
}
__device__ __forceinline__ unsigned int load_acquire(const unsigned int *p) {
    unsigned int v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// Waits (bounded) until the generation reaches `target`; the word behind it goes to *next.
__device__ __forceinline__ bool grid_wait(const unsigned int *gen, unsigned int target, unsigned int *next = nullptr) {
    const unsigned long long t0 = globaltimer_ns();
    for (uint32_t spin = 1;; ++spin) {
        unsigned int now;
        if (next) {
            unsigned long long both;
            asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(both) : "l"(gen) : "memory");
            now = static_cast<unsigned int>(both);
            *next = static_cast<unsigned int>(both >> 32);
        } else {
            now = load_acquire(gen);
        }
        if (static_cast<int>(now - target) >= 0) return true;
        if ((spin & 63u) == 0u && globaltimer_ns() - t0 > kWaitLimitNs) {
            raise_fault(kFaultTimeout);
            return false;
        }
    }
}

// 2^k that a row is divided by whose largest value past half's range has these bits: it comes
// below 2^15.
__device__ __forceinline__ int wide_exponent(unsigned int bits) { return static_cast<int>(bits >> 23) - 127 - 14; }
__device__ __forceinline__ float power_of_two(int k) { return __uint_as_float(static_cast<unsigned>(127 + k) << 23); }

// ---- step 1: scores ---------------------------------------------------------------------------------
// This lane's share of a dot product: chunks of 8 values first, first + step, ...; eight chunks of
// each row are under way at once where 16-byte loads are possible.
template <typename T>
__device__ __forceinline__ float dot_share(const uint16_t *x, const uint16_t *w, int D, int first, int step) {
    using H = Half16<T>;
    const int chunks = (D + 7) / 8;
    float s = 0.0f;
    auto add = [&](const uint4 &a, const uint4 &b, int count) {
        const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 fa = H::widen2(av[i]), fb = H::widen2(bv[i]);
            if (2 * i < count) s = fmaf(fa.x, fb.x, s);
            if (2 * i + 1 < count) s = fmaf(fa.y, fb.y, s);
        }
    };
    if (D % 8 == 0 && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(w)) & 15u) == 0) {
        const uint4 *xv = reinterpret_cast<const uint4 *>(x), *wv = reinterpret_cast<const uint4 *>(w);
        for (int c = first; c < chunks; c += 8 * step) {
            uint4 a[8], b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i * step < chunks) {
                    a[i] = __ldg(xv + c + i * step);
                    b[i] = __ldg(wv + c + i * step);
                }
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (c + i * step < chunks) add(a[i], b[i], 8);
        }
    } else {
        for (int c = first; c < chunks; c += step) {
            const int count = min(8, D - 8 * c);
            add(load8_any(x + 8 * c, count), load8_any(w + 8 * c, count), count);
        }
    }
    return s;
}

// Every CTA for itself when there is a score per warp at most (`local`): the grid barrier that
// would collect them costs about as much as they do. Otherwise an expert and 8 tokens per CTA, a
// warp per token (for fewer than 8 tokens, several warps share one token's D and their sums are
// added in a fixed order).
__host__ __device__ inline bool scores_local(const Moe16 &m) { return m.T * m.E <= 8; }

template <typename T, int THREADS>
__device__ __forceinline__ void moe_scores(const MoeParams &p, float *part, float *local) {
    const Moe16 &m = p.m;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp >= 8 && scores_local(m)) return;
    if (scores_local(m)) {
        if (warp < m.T * m.E) {
            const int t = warp / m.E, e = warp - t * m.E;
            float s = 0.0f;
            if (!(m.active && !m.active[t]))
                s = dot_share<T>(m.X + t * m.ldx, m.Wr + e * m.ldr, m.D, lane, 32);
            for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
            if (lane == 0) local[warp] = s;
        }
        return;
    }
    const int slices = m.T >= 8 ? 1 : m.T >= 4 ? 2 : m.T >= 2 ? 4 : 8;
    const int slice = warp & (slices - 1), t_step = 8 / slices;
    const int groups = (m.T + t_step - 1) / t_step;
    for (int item = blockIdx.x; item < m.E * groups; item += gridDim.x) {
        const int e = item / groups, t = (item - e * groups) * t_step + warp / slices;
        float s = 0.0f;
        const bool mine = warp < 8 && t < m.T;
        if (mine && !(m.active && !m.active[t]))
            s = dot_share<T>(m.X + t * m.ldx, m.Wr + e * m.ldr, m.D, slice * 32 + lane, slices * 32);
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
        if (slices > 1) {
            if (lane == 0 && warp < 8) part[warp] = s;
            __syncthreads();
            s = 0.0f;
            if (mine)
                for (int i = 0; i < slices; ++i) s += part[(warp & ~(slices - 1)) + i];
            __syncthreads();
        }
        if (lane == 0 && slice == 0 && mine) __stcg(p.score + t * m.E + e, s);
    }
}

// ---- step 2: routing ----------------------------------------------------------------------------------
// A warp per token, an expert's score in the registers of lane e % 32. Each chosen expert takes one
// warp-wide maximum of the scores and one minimum of the indices that have it.
template <int THREADS>
__device__ __forceinline__ void moe_route(const MoeParams &p, Routing &r, const float *local) {
    const Moe16 &m = p.m;
    constexpr int REGS = kMoeMaxExperts / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < m.E; e += THREADS) r.mask[e] = 0;
    __syncthreads();
    for (int t = warp; t < m.T; t += THREADS / 32) {
        if (m.active && !m.active[t]) {
            if (lane < m.k) {
                r.expert[t * m.k + lane] = kNone;
                r.weight[t * m.k + lane] = 0.0f;
                if (blockIdx.x == 0 && m.index) m.index[t * m.k + lane] = -1;
                if (blockIdx.x == 0 && m.weight) m.weight[t * m.k + lane] = 0.0f;
            }
            continue;
        }
        unsigned int key[REGS];  // 0, below every score, where there is no expert or none any more
        unsigned int best = 0;
#pragma unroll
        for (int i = 0; i < REGS; ++i) {
            const int e = i * 32 + lane;
            key[i] = 0u;
            if (i * 32 < m.E && e < m.E)
                key[i] = moe_score_order(local ? local[t * m.E + e] : __ldcg(p.score + t * m.E + e));
        }
#pragma unroll
        for (int i = 0; i < REGS; ++i) best = max(best, key[i]);
        const float top = moe_order_score(__reduce_max_sync(0xFFFFFFFFu, best));
        float sum = 0.0f;  // of every expert's exp(s - top), or of the chosen ones'
        if (!m.renormalize) {
#pragma unroll
            for (int i = 0; i < REGS; ++i)
                if (i * 32 + lane < m.E) sum += expf(moe_order_score(key[i]) - top);
        }
        int chosen = -1;  // lane j keeps the j-th
        float w = 0.0f;
        for (int j = 0; j < m.k; ++j) {
            unsigned int high = 0;
            int at = 0x7FFFFFFF;
#pragma unroll
            for (int i = 0; i < REGS; ++i)
                if (key[i] > high) {
                    high = key[i];
                    at = i * 32 + lane;
                }
            const unsigned int win = __reduce_max_sync(0xFFFFFFFFu, high);
            const int e = __reduce_min_sync(0xFFFFFFFFu, high == win ? at : 0x7FFFFFFF);
            if (lane == j) {
                chosen = e;
                w = expf(moe_order_score(win) - top);
            }
            if (lane == (e & 31)) {
#pragma unroll
                for (int i = 0; i < REGS; ++i)
                    if (i == e >> 5) key[i] = 0u;
            }
        }
        if (m.renormalize) sum = w;
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        if (lane < m.k) {
            w = w / sum;
            r.expert[t * m.k + lane] = static_cast<uint16_t>(chosen);
            r.weight[t * m.k + lane] = w;
            atomicOr(reinterpret_cast<unsigned int *>(&r.mask[chosen]) + (t >> 5), 1u << (t & 31));
            if (blockIdx.x == 0 && m.index) m.index[t * m.k + lane] = chosen;
            if (blockIdx.x == 0 && m.weight) m.weight[t * m.k + lane] = w;
        }
    }
    __syncthreads();
    if (warp == 0) {
        int rows = 0, n = 0;
        for (int e0 = 0; e0 < m.E; e0 += 32) {
            const int e = e0 + lane;
            const int c = e < m.E ? __popcll(r.mask[e]) : 0;
            int scan = c;
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xFFFFFFFFu, scan, o);
                if (lane >= o) scan += v;
            }
            const unsigned int used = __ballot_sync(0xFFFFFFFFu, c > 0);
            if (c > 0) {
                const int at = n + __popc(used & ((1u << lane) - 1u));
                r.offset[e] = static_cast<uint16_t>(rows + scan - c);
                r.rank[e] = static_cast<uint16_t>(at);
                r.active[at] = static_cast<uint16_t>(e);
            }
            rows += __shfl_sync(0xFFFFFFFFu, scan, 31);
            n += __popc(used);
        }
        if (lane == 0) r.n_active = n;
    }
    __syncthreads();
}

template <int NT, bool GATED, typename T>
__global__ void __launch_bounds__((MoeConfig<NT, GATED>::THREADS), 1)
    moe_stream_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_g,
                      const __grid_constant__ CUtensorMap map_u, const __grid_constant__ CUtensorMap map_d,
                      const __grid_constant__ CUtensorMap map_h, const MoeParams p) {
    using C = MoeConfig<NT, GATED>;
    using H = Half16<T>;
    constexpr int STAGES = C::STAGES, ACCS = C::ACCS;
    const Moe16 &m = p.m;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t pad = (1024u - (smem_addr(smem_raw) & 1023u)) & 1023u;
    uint8_t *smem = smem_raw + pad;
    Routing &route = *reinterpret_cast<Routing *>(smem + STAGES * C::STAGE_BYTES);
    uint64_t *full = reinterpret_cast<uint64_t *>(
        smem + STAGES * C::STAGE_BYTES + (sizeof(Routing) + 7) / 8 * 8);
    uint64_t *empty = full + STAGES;
    uint64_t *acc_full = empty + STAGES;  // [2]
    uint64_t *acc_free = acc_full + 2;    // [2]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_free + 2);
    float *part = reinterpret_cast<float *>(tmem_slot + 2);  // [8]
    unsigned int *gen_slot = tmem_slot + 10;  // the barriers' generation before step 3's
    unsigned int *wide_slot = tmem_slot + 11;
    uint64_t *gate = reinterpret_cast<uint64_t *>(tmem_slot + 12);  // half: h is complete and in range
    constexpr bool RANGE = H::kind == kF16;  // h may be past its type's range
    const bool local = scores_local(m);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const unsigned int ctas = gridDim.x;
    unsigned int gen0 = 0;
    if (threadIdx.x == 0) {
        gen0 = load_acquire(&p.sync->gen);  // read before this CTA's first arrival
        *gen_slot = gen0;
        *wide_slot = 0;
        tma_prefetch_desc(&map_x);
        if (GATED) tma_prefetch_desc(&map_g);
        tma_prefetch_desc(&map_u);
        tma_prefetch_desc(&map_d);
        tma_prefetch_desc(&map_h);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int j = 0; j < 2; ++j) {
            mbar_init(&acc_full[j], 1);
            mbar_init(&acc_free[j], 4 * C::GROUPS);
        }
        mbar_init(gate, 1);
        mbar_init_fence();
    }
    if (warp == 2) tmem_alloc<1>(tmem_slot, C::TMEM_COLS);
    moe_scores<T, C::THREADS>(p, part, part);
    tc_before_sync();
    __syncthreads();
    tc_after_sync();
    const uint32_t tmem = *tmem_slot;
    if (!local) {
        if (threadIdx.x == 0) {
            grid_arrive(&p.sync->count[0], &p.sync->gen, ctas);
            grid_wait(&p.sync->gen, ++gen0);
            *gen_slot = gen0;
        }
        __syncthreads();
    }
    moe_route<C::THREADS>(p, route, local ? part : nullptr);
    const int n_active = route.n_active;
    UnitSplit up, down;
    up.total = n_active * p.tiles_f * p.kb_up;
    up.ctas = min(static_cast<int>(ctas), max(up.total / min_run(NT), min(n_active * p.tiles_f, static_cast<int>(ctas))));
    down.total = n_active * p.tiles_d * p.kb_down;
    down.ctas = min(static_cast<int>(ctas), max(down.total / min_run(NT), min(n_active * p.tiles_d, static_cast<int>(ctas))));
    const int cta = blockIdx.x;
    const int up0 = cta < up.ctas ? up.first(cta) : 0, up1 = cta < up.ctas ? up.first(cta + 1) : 0;
    const int dn0 = cta < down.ctas ? down.first(cta) : 0, dn1 = cta < down.ctas ? down.first(cta + 1) : 0;

    if (warp == 0) {
        if (lane == 0) {
            RingCursor<STAGES> ring;
            int issued = 0;
            bool ok = true;
            int tile = p.kb_up ? up0 / p.kb_up : 0, kb = up0 - tile * p.kb_up;
            for (int u = up0; u < up1 && ok; ++u) {
                if (issued >= STAGES && !mbar_wait(&empty[ring.stage], ring.parity ^ 1u)) {
                    ok = false;
                    break;
                }
                uint8_t *sw = smem + ring.stage * C::STAGE_BYTES, *sx = sw + C::A_BYTES;
                uint64_t *bar = &full[ring.stage];
                mbar_arrive_expect_tx(bar, C::STAGE_BYTES);
                const int e = route.active[tile / p.tiles_f], f0 = tile % p.tiles_f * kStreamRows;
                if (GATED) tma_load_3d(sw, &map_g, bar, kb * kStreamK, f0, e);
                tma_load_3d(sw + (ACCS - 1) * C::W_BYTES, &map_u, bar, kb * kStreamK, f0, e);
                tma_load_2d(sx, &map_x, bar, kb * kStreamK, 0);
                ring.next();
                ++issued;
                if (++kb == p.kb_up) {
                    kb = 0;
                    ++tile;
                }
            }
            // Step 4: the weights of the first stages, then the barrier, then their rows of h.
            RingCursor<STAGES> behind = ring;
            int waiting = 0;
            bool open = false;
            tile = p.kb_down ? dn0 / p.kb_down : 0;
            kb = dn0 - tile * p.kb_down;
            int tile_h = tile, kb_h = kb;
            auto load_rows = [&]() {
                const int e = route.active[tile_h / p.tiles_d];
                tma_load_2d(smem + behind.stage * C::STAGE_BYTES + C::A_BYTES, &map_h, &full[behind.stage],
                            kb_h * kStreamK, route.offset[e]);
                behind.next();
                if (++kb_h == p.kb_down) {
                    kb_h = 0;
                    ++tile_h;
                }
            };
            auto open_gate = [&]() {
                ok = (RANGE ? mbar_wait(gate, 0) : grid_wait(&p.sync->gen, gen0 + 1)) && ok;
                asm volatile("fence.proxy.async;" ::: "memory");  // h was written by plain stores
                open = true;
                for (; waiting > 0; --waiting) load_rows();
            };
            for (int u = dn0; u < dn1 && ok; ++u) {
                if (!open && waiting == STAGES) open_gate();
                if (issued >= STAGES && !mbar_wait(&empty[ring.stage], ring.parity ^ 1u)) {
                    ok = false;
                    break;
                }
                uint8_t *sw = smem + ring.stage * C::STAGE_BYTES;
                uint64_t *bar = &full[ring.stage];
                mbar_arrive_expect_tx(bar, C::W_BYTES + C::X_BYTES);
                const int e = route.active[tile / p.tiles_d], d0 = tile % p.tiles_d * kStreamRows;
                tma_load_3d(sw, &map_d, bar, kb * kStreamK, d0, e);
                ring.next();
                ++issued;
                if (++kb == p.kb_down) {
                    kb = 0;
                    ++tile;
                }
                if (open)
                    load_rows();
                else
                    ++waiting;
            }
            if (waiting > 0) open_gate();
            // Shared memory must outlive every copy: wait (bounded) for the last stages.
            for (int j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
                if (!mbar_wait(&full[j % STAGES], (j / STAGES) & 1)) break;
        }
    } else if (warp == 1) {
        if (lane == 0) {
            RingCursor<STAGES> ring;
            int j = -1;
            bool ok = true;
            uint32_t d = tmem;
#pragma unroll 1
            for (int step = 0; step < 2; ++step) {
                const int KB = step ? p.kb_down : p.kb_up, u0 = step ? dn0 : up0, u1 = step ? dn1 : up1;
                int kb = u1 > u0 ? u0 % KB : 0;
                for (int u = u0; u < u1 && ok; ++u) {
                    const bool first = u == u0 || kb == 0;
                    if (first) {
                        ++j;
                        if (j >= 2 && !mbar_wait(&acc_free[j & 1], ((j >> 1) - 1) & 1)) {
                            ok = false;
                            break;
                        }
                        tc_after_sync();
                        d = tmem + static_cast<uint32_t>((j & 1) * ACCS * NT);
                    }
                    if (!mbar_wait(&full[ring.stage], ring.parity)) {
                        ok = false;
                        break;
                    }
                    tc_after_sync();
                    const uint32_t sw = smem_addr(smem + ring.stage * C::STAGE_BYTES);
                    const uint64_t dx = desc_k_major(sw + C::A_BYTES);
                    const int accs = step ? 1 : ACCS;
#pragma unroll
                    for (int a = 0; a < ACCS; ++a) {
                        if (a >= accs) break;
                        const uint64_t dw = desc_k_major(sw + a * C::W_BYTES);
#pragma unroll
                        for (int k = 0; k < kStreamK / 16; ++k)
                            mma_16<1>(d + static_cast<uint32_t>(a * NT), dw + static_cast<uint64_t>(2 * k),
                                      dx + static_cast<uint64_t>(2 * k), p.idesc, !first || k > 0);
                    }
                    mma_commit_16<1>(&empty[ring.stage]);
                    ring.next();
                    if (++kb == KB) kb = 0;
                    if (kb == 0 || u + 1 == u1) mma_commit_16<1>(&acc_full[j & 1]);
                }
            }
        }
    } else if (warp >= 4) {
        const int row = (warp & 3) * 32 + lane;
        const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
        constexpr int COLS = NT / C::GROUPS;
        const int first_col = (warp - 4) / 4 * COLS, end_col = first_col + COLS;
        int j = 0;
        bool ok = true;  // after a wait that expired the loops run on without waiting, so that
                         // every warp still meets the others at the barrier below
        // h of expert e, hidden value f, tokens c .. c + 15
        auto emit = [&](int e, int f, int c, const float(&g)[16], const float(&v)[16]) {
            const unsigned long long mask = route.mask[e];
            float x[16];
            with_activation(m.act, [&](auto a) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    x[i] = GATED ? activate16<decltype(a)::value>(g[i]) * v[i]
                                 : activate16<decltype(a)::value>(v[i]);
            });
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (!((mask >> (c + i)) & 1ull) || f >= m.F) continue;
                const int slot = route.offset[e] + __popcll(mask & ((1ull << (c + i)) - 1ull));
                const uint16_t v16 = H::narrow(x[i]);
                p.h[slot * p.ldh + f] = v16;
                if (RANGE && (v16 & 0x7FFFu) == 0x7C00u) {
                    p.wide[static_cast<long long>(slot) * m.F + f] = x[i];
                    if (fabsf(x[i]) < INFINITY) {
                        atomicMax(&p.sync->largest[slot], __float_as_uint(fabsf(x[i])));
                        atomicExch(&p.sync->wide, 1u);
                    }
                }
            }
        };
        for (int u = up0; u < up1; ++j) {
            const int tile = u / p.kb_up, kb0 = u - tile * p.kb_up;
            const int n_units = min(p.kb_up - kb0, up1 - u);
            u += n_units;
            ok = ok && mbar_wait(&acc_full[j & 1], (j >> 1) & 1);
            tc_after_sync();
            const uint32_t acc = tmem + lane_base + static_cast<uint32_t>((j & 1) * ACCS * NT);
            const int e = route.active[tile / p.tiles_f], f = tile % p.tiles_f * kStreamRows + row;
            const unsigned long long mask = route.mask[e];
            const bool whole = n_units == p.kb_up;
            const int slot = (2 * cta + (kb0 == 0 ? 1 : 0)) * ACCS;
#pragma unroll 1
            for (int c = first_col; c < end_col; c += 16) {
                uint32_t r[ACCS][16];
#pragma unroll
                for (int a = 0; a < ACCS; ++a) tmem_ld_x16(acc + static_cast<uint32_t>(a * NT + c), r[a]);
                tmem_ld_wait();
                if (c + 16 == end_col) {
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[j & 1]);
                }
                if (!((mask >> c) & 0xFFFFull)) continue;
                if (whole) {
                    float g[16], v[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        g[i] = __uint_as_float(r[0][i]);
                        v[i] = __uint_as_float(r[ACCS - 1][i]);
                    }
                    emit(e, f, c, g, v);
                } else {
#pragma unroll
                    for (int a = 0; a < ACCS; ++a) put_piece<NT>(p.up_pieces, slot + a, c, row, m.T, r[a]);
                }
            }
            if (whole || !piece_arrived(p.counters + static_cast<size_t>(tile) * (4 * C::GROUPS) + warp - 4, n_units, p.kb_up, lane))
                continue;
            const int c0 = up.owner(tile * p.kb_up), c1 = up.owner(tile * p.kb_up + p.kb_up - 1);
#pragma unroll 1
            for (int c = first_col; c < end_col; c += 16) {
                if (!((mask >> c) & 0xFFFFull)) continue;
                float g[16], v[16];
                sum_pieces<NT>(p.up_pieces, c0, c1, ACCS, ACCS - 1, c, row, m.T, v);
                if (GATED)
                    sum_pieces<NT>(p.up_pieces, c0, c1, ACCS, 0, c, row, m.T, g);
                emit(e, f, c, g, v);
            }
        }
        // This CTA's part of h is written: step 4 may read it through the async proxy.
        asm volatile("fence.proxy.async;" ::: "memory");
        __threadfence();
        asm volatile("bar.sync 1, %0;" ::"n"(128 * C::GROUPS) : "memory");  // the epilogue's warps
        if (threadIdx.x == 128) grid_arrive(&p.sync->count[1], &p.sync->gen, ctas);
        if (RANGE) {
            if (threadIdx.x == 128) {
                unsigned int flag = 0;
                grid_wait(&p.sync->gen, *gen_slot + 1, &flag);
                *wide_slot = flag;
                if (!flag) mbar_arrive(gate);
            }
            asm volatile("bar.sync 1, %0;" ::"n"(128 * C::GROUPS) : "memory");
            if (*wide_slot) {
                for (int slot = 0; slot < m.T * m.k; ++slot) {
                    const unsigned int bits = __ldcg(&p.sync->largest[slot]);
                    if (bits == 0) continue;
                    const float factor = power_of_two(-wide_exponent(bits));
                    for (int f = cta * (128 * C::GROUPS) + threadIdx.x - 128; f < m.F; f += ctas * (128 * C::GROUPS)) {
                        uint16_t *v = p.h + slot * p.ldh + f;
                        const uint16_t v16 = __ldcg(v);
                        const float x = (v16 & 0x7FFFu) == 0x7C00u ? __ldcg(p.wide + static_cast<long long>(slot) * m.F + f)
                                                                   : H::widen(v16);
                        *v = H::narrow(x * factor);
                    }
                }
                asm volatile("fence.proxy.async;" ::: "memory");
                __threadfence();
                asm volatile("bar.sync 1, %0;" ::"n"(128 * C::GROUPS) : "memory");
                if (threadIdx.x == 128) {
                    grid_arrive(&p.sync->count[3], &p.sync->gen, ctas);
                    grid_wait(&p.sync->gen, *gen_slot + 2);
                    mbar_arrive(gate);
                }
            }
        }
        const long long ldo = static_cast<long long>(p.tiles_d) * kStreamRows;
        for (int u = dn0; u < dn1; ++j) {
            const int tile = u / p.kb_down, kb0 = u - tile * p.kb_down;
            const int n_units = min(p.kb_down - kb0, dn1 - u);
            u += n_units;
            ok = ok && mbar_wait(&acc_full[j & 1], (j >> 1) & 1);
            tc_after_sync();
            const uint32_t acc = tmem + lane_base + static_cast<uint32_t>((j & 1) * ACCS * NT);
            const int e = route.active[tile / p.tiles_d], rows = __popcll(route.mask[e]);
            const bool whole = n_units == p.kb_down;
            float *dst = p.out + route.offset[e] * ldo + tile % p.tiles_d * kStreamRows + row;
#pragma unroll 1
            for (int c = first_col; c < end_col; c += 16) {
                uint32_t r[16];
                tmem_ld_x16(acc + static_cast<uint32_t>(c), r);
                tmem_ld_wait();
                if (c + 16 == end_col) {
                    tc_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&acc_free[j & 1]);
                }
                if (whole) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < rows) __stcg(dst + (c + i) * ldo, __uint_as_float(r[i]));
                } else {
                    float *piece = p.down_pieces +
                                   static_cast<size_t>(2 * cta + (kb0 == 0 ? 1 : 0)) * NT * kStreamRows + row;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (c + i < rows) __stcg(piece + (c + i) * kStreamRows, __uint_as_float(r[i]));
                }
            }
        }
    }

    // ---- the sum over each token's experts -----------------------------------------------------------
    __syncwarp();
    __threadfence();
    tc_before_sync();
    __syncthreads();
    const bool wide = RANGE && *wide_slot != 0;
    if (threadIdx.x == 0) {
        grid_arrive(&p.sync->count[2], &p.sync->gen, ctas);
        grid_wait(&p.sync->gen, gen0 + (wide ? 3 : 2));
    }
    __syncthreads();
    if (warp == 2) {
        tc_after_sync();
        tmem_dealloc<1>(tmem, C::TMEM_COLS);
    }
    const long long ldo = static_cast<long long>(p.tiles_d) * kStreamRows;
    // A warp takes 128 features of one token, four per lane; lane j finds where its j-th expert's
    // output lies (a whole tile's in `out`, a cut one's in pieces first .. last).
    constexpr int WARPS = C::THREADS / 32;
    const long long items = static_cast<long long>(m.T) * p.tiles_d;
    for (long long i = blockIdx.x * WARPS + warp; i < items; i += ctas * WARPS) {
        const int t = static_cast<int>(i / p.tiles_d), tile_d = static_cast<int>(i - static_cast<long long>(t) * p.tiles_d);
        const int d = tile_d * kStreamRows + 4 * lane, count = min(4, m.D - d);
        float y[4] = {}, res[4] = {};
        if (m.R)
#pragma unroll
            for (int v = 0; v < 4; ++v)
                if (v < count) res[v] = H::widen(m.R[t * m.ldres + d + v]);
        int col = 0, first = -1, last = -1, out_row = 0;
        float scale = 1.0f;  // what the expert's row of h was divided by
        const int e = lane < m.k ? route.expert[t * m.k + lane] : kNone;
        if (e != kNone) {
            col = __popcll(route.mask[e] & ((1ull << t) - 1ull));
            out_row = route.offset[e] + col;
            const int unit = (route.rank[e] * p.tiles_d + tile_d) * p.kb_down;
            first = down.owner(unit);
            last = down.owner(unit + p.kb_down - 1);
            if (wide) {
                const unsigned int bits = __ldcg(&p.sync->largest[out_row]);
                if (bits) scale = power_of_two(wide_exponent(bits));
            }
        }
        auto piece = [&](int slot, int c) {
            return __ldcg(reinterpret_cast<const float4 *>(
                p.down_pieces + (static_cast<size_t>(slot) * NT + c) * kStreamRows + 4 * lane));
        };
        const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        // Four experts' values under way at once, in up to two pieces each; more pieces are rare.
        for (int j0 = 0; j0 < m.k; j0 += 4) {
            float4 a[4], b[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {  // m.k is at most 16: a lane of its own for each
                const int c0 = __shfl_sync(0xFFFFFFFFu, first, j0 + q), c1 = __shfl_sync(0xFFFFFFFFu, last, j0 + q);
                const int cj = __shfl_sync(0xFFFFFFFFu, col, j0 + q), rj = __shfl_sync(0xFFFFFFFFu, out_row, j0 + q);
                a[q] = c0 < 0 ? zero
                       : c0 == c1 ? __ldcg(reinterpret_cast<const float4 *>(p.out + rj * ldo + d))
                                  : piece(2 * c0 + 1, cj);
                b[q] = c0 < c1 ? piece(2 * (c0 + 1), cj) : zero;
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c0 = __shfl_sync(0xFFFFFFFFu, first, j0 + q), c1 = __shfl_sync(0xFFFFFFFFu, last, j0 + q);
                const int cj = __shfl_sync(0xFFFFFFFFu, col, j0 + q);
                if (c0 < 0) continue;
                float4 s = make_float4(a[q].x + b[q].x, a[q].y + b[q].y, a[q].z + b[q].z, a[q].w + b[q].w);
                for (int k = c0 + 2; k <= c1; ++k) {
                    const float4 x = piece(2 * k, cj);
                    s.x += x.x;
                    s.y += x.y;
                    s.z += x.z;
                    s.w += x.w;
                }
                float w = route.weight[t * m.k + j0 + q];
                if (RANGE && wide) w *= __shfl_sync(0xFFFFFFFFu, scale, j0 + q);
                y[0] = fmaf(w, s.x, y[0]);
                y[1] = fmaf(w, s.y, y[1]);
                y[2] = fmaf(w, s.z, y[2]);
                y[3] = fmaf(w, s.w, y[3]);
            }
        }
#pragma unroll
        for (int v = 0; v < 4; ++v)
            if (v < count) m.Y[t * m.ldy + d + v] = H::narrow(y[v] + res[v]);
    }
    if (RANGE && wide) {  // the last CTA to get here leaves zeros for the next call
        __syncthreads();
        if (threadIdx.x == 0) *wide_slot = atomicAdd(&p.sync->done, 1u);
        __syncthreads();
        if (*wide_slot == ctas - 1) {
            for (int slot = threadIdx.x; slot < m.T * m.k; slot += C::THREADS) p.sync->largest[slot] = 0;
            if (threadIdx.x == 0) p.sync->wide = p.sync->done = 0;
        }
    }
}

// ---- host side ------------------------------------------------------------------------------------------

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

template <int NT, bool GATED, typename T>
cudaError_t launch(const Moe16 &m, cudaStream_t stream, const char **detail) {
    using C = MoeConfig<NT, GATED>;
    static_assert(C::SMEM <= 227 * 1024 && C::STAGES >= 3, "ring and routing fit in shared memory");
    auto kernel = moe_stream_kernel<NT, GATED, T>;
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
        *detail = "mixture-of-experts kernel set-up failed";
        return setup[dev];
    }
    MoeParams p;
    p.m = m;
    p.tiles_f = static_cast<int>((m.F + static_cast<long long>(kStreamRows) - 1) / kStreamRows);
    p.kb_up = static_cast<int>((m.D + static_cast<long long>(kStreamK) - 1) / kStreamK);
    p.tiles_d = static_cast<int>((m.D + static_cast<long long>(kStreamRows) - 1) / kStreamRows);
    p.kb_down = static_cast<int>((m.F + static_cast<long long>(kStreamK) - 1) / kStreamK);
    p.idesc = idesc_16(kStreamRows, NT, Half16<T>::kind, false, false);
    const size_t pairs = static_cast<size_t>(m.T) * m.k, G = static_cast<size_t>(sms[dev]);
    const size_t experts = std::min<size_t>(m.E, pairs);
    void *sync = nullptr, *data = nullptr;
    err = layer_scratch(kScratchMoeSync, stream, kSyncBytes + experts * p.tiles_f * 16 * C::GROUPS, &sync, detail);
    if (err != cudaSuccess) return err;
    p.sync = static_cast<MoeSync *>(sync);
    p.counters = reinterpret_cast<unsigned int *>(static_cast<char *>(sync) + kSyncBytes);
    p.ldh = (m.F + 7LL) / 8 * 8;
    const size_t b_score = round256(static_cast<size_t>(m.T) * m.E * 4);
    const size_t b_h = round256(pairs * p.ldh * 2);
    const size_t b_out = round256(pairs * p.tiles_d * kStreamRows * 4);
    const size_t b_wide = Half16<T>::kind == kF16 ? round256(pairs * m.F * 4) : 0;
    const size_t b_up = 2 * G * C::ACCS * NT * kStreamRows * 4, b_down = 2 * G * NT * kStreamRows * 4;
    err = layer_scratch(kScratchMoe, stream, b_score + b_h + b_wide + b_out + b_up + b_down, &data, detail);
    if (err != cudaSuccess) return err;
    char *at = static_cast<char *>(data);
    p.score = reinterpret_cast<float *>(at);
    p.h = reinterpret_cast<uint16_t *>(at += b_score);
    p.wide = reinterpret_cast<float *>(at += b_h);
    p.out = reinterpret_cast<float *>(at += b_wide);
    p.up_pieces = reinterpret_cast<float *>(at += b_out);
    p.down_pieces = reinterpret_cast<float *>(at += b_up);

    const long long su = m.E > 1 ? m.su : m.F * m.ldu, sd = m.E > 1 ? m.sd : m.D * m.ldd;
    CUtensorMap mx, mg, mu, md, mh;
    if (!tensor_map_16(&mx, m.X, m.dtype, m.D, m.T, m.ldx, kStreamK, NT) ||
        (GATED && !tensor_map_16(&mg, m.Wg, m.dtype, m.D, m.F, m.ldu, kStreamK, kStreamRows, false, m.E, su)) ||
        !tensor_map_16(&mu, m.Wu, m.dtype, m.D, m.F, m.ldu, kStreamK, kStreamRows, false, m.E, su) ||
        !tensor_map_16(&md, m.Wd, m.dtype, m.F, m.D, m.ldd, kStreamK, kStreamRows, false, m.E, sd) ||
        !tensor_map_16(&mh, p.h, m.dtype, m.F, static_cast<long long>(pairs), p.ldh, kStreamK, NT)) {
        *detail = "cuTensorMapEncodeTiled rejected a matrix";
        return cudaErrorInvalidValue;
    }
    if (!GATED) mg = mu;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(G), 1, 1);
    cfg.blockDim = dim3(C::THREADS, 1, 1);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeCooperative;  // the grid barriers need every CTA resident
    attr[0].val.cooperative = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    err = cudaLaunchKernelEx(&cfg, kernel, mx, mg, mu, md, mh, p);
    if (err == cudaSuccess) err = cudaGetLastError();
    if (err != cudaSuccess) *detail = "mixture-of-experts kernel launch failed";
    return err;
}

template <int NT, typename T>
cudaError_t launch_gate(const Moe16 &m, cudaStream_t stream, const char **detail) {
    return m.Wg ? launch<NT, true, T>(m, stream, detail) : launch<NT, false, T>(m, stream, detail);
}
template <typename T>
cudaError_t launch_width(const Moe16 &m, cudaStream_t stream, const char **detail) {
    if (m.T <= 16) return launch_gate<16, T>(m, stream, detail);
    if (m.T <= 32) return launch_gate<32, T>(m, stream, detail);
    return launch_gate<64, T>(m, stream, detail);
}

}  // namespace

bool moe_stream_supports(const Moe16 &m) {
    if (m.D == 0 || m.F == 0) return false;
    const long long e = std::min<long long>(m.E, static_cast<long long>(m.T) * m.k);
    const long long up = e * ((m.F + 127LL) / 128) * ((m.D + 63LL) / 64);
    const long long down = e * ((m.D + 127LL) / 128) * ((m.F + 63LL) / 64);
    return up <= 0x7fffffffLL && down <= 0x7fffffffLL && tma_rows(m.X, m.ldx) && tma_rows(m.Wu, m.ldu) &&
           (!m.Wg || tma_rows(m.Wg, m.ldu)) && tma_rows(m.Wd, m.ldd) && (m.E == 1 || (m.su % 8 == 0 && m.sd % 8 == 0));
}

cudaError_t moe_stream_launch(const Moe16 &m, cudaStream_t stream, const char **detail) {
    return m.dtype == kBf16 ? launch_width<__nv_bfloat16>(m, stream, detail)
                            : launch_width<__half>(m, stream, detail);
}

}  // namespace sg
