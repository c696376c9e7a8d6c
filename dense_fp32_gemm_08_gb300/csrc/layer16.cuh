// layer16.cuh: host-visible description of the 16-bit layer operators (linear layer, its
// gradients, mixture-of-experts layer), used by the C ABI in sgemm_api.cu.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace sg {

// One product D = act(A . B + bias) + res on 16-bit values (accumulated in fp32, each output
// rounded once), with pre = A . B + bias kept on request. A is M x K and B is K x N.
struct Gemm16 {
    int dtype = 0;  // Dtype16 (half16.cuh)
    int M = 0, N = 0, K = 0;
    const uint16_t *A = nullptr;
    long long lda = 0;
    bool a_mn = false;  // false: rows of A stored (K contiguous); true: A stored K x M
    const uint16_t *B = nullptr;
    long long ldb = 0;
    bool b_mn = false;  // false: B stored N x K (K contiguous); true: B stored K x N
    uint16_t *D = nullptr;
    long long ldd = 0;
    const uint16_t *bias = nullptr;  // N values
    int act = 0;                     // Activation (epilogue.cuh)
    const uint16_t *res = nullptr;
    long long ldr = 0;
    uint16_t *pre = nullptr;
    long long ldz = 0;
};

// True when TMA can address the matrix's rows: 16-byte aligned base and leading dimension.
inline bool tma_rows(const void *p, long long ld) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld % 8 == 0;
}

// Programmatic dependent launch: each kernel of the layer operators lets the stream's next one
// start its prologue early (grid_dependents) and touches global memory only after the kernels
// before it have completed (grid_dependency); set_early_start() asks for it at launch.
__device__ __forceinline__ void grid_dependents() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
inline void set_early_start(cudaLaunchAttribute &attr) {
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
}
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), dim3 grid, unsigned threads, size_t smem,
                         cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    set_early_start(attr[0]);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// One or two independent products; the larger kernels run them as one grid.
constexpr int kMaxProducts = 2;
cudaError_t gemm16_launch(const Gemm16 *list, int n, cudaStream_t stream, const char **detail);

// The elementwise part of the linear layer's gradient: dz = dy * act'(z), M x N, and its
// column sums db (fp32), either of them optional. dz == nullptr: only the sums.
struct ActGrad {
    int dtype = 0;
    int M = 0, N = 0;
    const uint16_t *dy = nullptr;
    long long lddy = 0;
    const uint16_t *z = nullptr;
    long long ldz = 0;
    int act = 0;
    uint16_t *dz = nullptr;
    long long lddz = 0;
    float *db = nullptr;
};

cudaError_t act_grad_launch(const ActGrad &g, cudaStream_t stream, const char **detail);

// A whole mixture-of-experts layer for T tokens.
struct Moe16 {
    int dtype = 0, act = 0;
    int T = 0, E = 0, k = 0, D = 0, F = 0;
    const uint16_t *X = nullptr;
    long long ldx = 0;
    const uint16_t *Wr = nullptr;
    long long ldr = 0;
    const uint16_t *Wg = nullptr, *Wu = nullptr;  // Wg == nullptr: no gate
    long long ldu = 0, su = 0;
    const uint16_t *Wd = nullptr;
    long long ldd = 0, sd = 0;
    bool renormalize = false;
    const uint8_t *active = nullptr;
    const uint16_t *R = nullptr;
    long long ldres = 0;
    uint16_t *Y = nullptr;
    long long ldy = 0;
    int *index = nullptr;
    float *weight = nullptr;
};

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopk = 16;

cudaError_t moe16_launch(const Moe16 &m, cudaStream_t stream, const char **detail);

// Per-(device, stream) scratch of the layer operators, one buffer per use. Grown when a call
// needs more; buffers and the ones they outgrew are kept until release_layer_workspaces().
enum LayerScratch : int {
    kScratchDz = 0,    // the gradient's dz
    kScratchSums = 1,  // partial column sums
    kScratchMoe = 2,   // scores, hidden values and partial sums of the mixture of experts
    kScratchPack = 3,  // aligned copies of operands TMA cannot address
    kScratchStream = 4,  // arrival counters and partial tiles of the weight-streaming product
    kScratchMoeSync = 5,  // its barriers and arrival counters
    kScratchSumSync = 6,  // arrival counters of the column sums
    kScratchPair = 7,      // pieces of the pair product's cut tiles
    kScratchPairSync = 8,  // their arrival counters
    kScratchUses
};
cudaError_t layer_scratch(LayerScratch use, cudaStream_t stream, size_t bytes, void **out,
                          const char **detail);
cudaError_t release_layer_workspaces();
// After a bounded wait expired: counters left by the kernel that gave up are cleared (in stream
// order) before each scratch buffer's next use.
void layer_scratch_distrust();

}  // namespace sg
