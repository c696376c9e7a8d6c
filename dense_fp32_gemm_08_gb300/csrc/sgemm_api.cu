// sgemm_api.cu: the C ABI (include/sgemm.h): argument checks, fast exits, kernel choice and
// status reporting. Every compute step runs in the CUDA kernels of this library.
#include "sgemm.h"

#include <algorithm>
#include <atomic>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <mutex>
#include <vector>

#include "config_table.h"
#include "epilogue.cuh"
#include "host_gemm.cuh"
#include "layer16.cuh"
#include "ptx.cuh"
#include "simt_gemm.cuh"
#include "tf32x3_gemm.cuh"

namespace sg {
namespace {
std::mutex &fault_reader_mutex() {
    static std::mutex m;
    return m;
}
std::vector<FaultWordReader> &fault_readers() {
    static std::vector<FaultWordReader> v;
    return v;
}
}  // namespace

void register_fault_word_reader(FaultWordReader reader) {
    std::lock_guard<std::mutex> lock(fault_reader_mutex());
    fault_readers().push_back(reader);
}

unsigned int take_fault_words(cudaStream_t stream) {
    std::vector<FaultWordReader> readers;
    {
        std::lock_guard<std::mutex> lock(fault_reader_mutex());
        readers = fault_readers();
    }
    unsigned int word = 0;
    for (FaultWordReader read : readers) word |= read(stream);
    return word;
}
}  // namespace sg

namespace {

thread_local char t_last_error[256] = "";

sgemm_status_t fail(sgemm_status_t st, const char *what) {
    std::snprintf(t_last_error, sizeof(t_last_error), "%s", what);
    return st;
}

sgemm_status_t fail_cuda(const char *what, cudaError_t err) {
    std::snprintf(t_last_error, sizeof(t_last_error), "%s: %s", what, cudaGetErrorString(err));
    return SGEMM_ERR_LAUNCH;
}

constexpr long long kMaxDim = 0x7fffffffLL;  // kernels index M, N, K with 32-bit ints

std::atomic<int> g_forced_config{-2};  // -2: environment not read yet, -1: automatic

int forced_config() {
    int v = g_forced_config.load(std::memory_order_relaxed);
    if (v == -2) {
        const char *env = std::getenv("SGEMM_FORCE_CONFIG");
        int want = -1;
        if (env && *env) {
            char *end = nullptr;
            long id = std::strtol(env, &end, 10);
            if (end && *end == '\0' && id >= 0 && id < sg::simt_num_configs()) want = (int)id;
        }
        int expected = -2;
        g_forced_config.compare_exchange_strong(expected, want);
        v = g_forced_config.load(std::memory_order_relaxed);
    }
    return v;
}

bool log_enabled() {
    static const bool on = [] {
        const char *env = std::getenv("SGEMM_LOG");
        return env && *env && std::strcmp(env, "0") != 0;
    }();
    return on;
}

// C = beta * C (zeros when beta == 0, C not read then), the whole product when alpha == 0 or
// K == 0; with a fused epilogue, C = act(bias) + beta * C. Rows over the grid's y dimension
// (batch entries stacked), columns over threads.
__global__ void scale_c_kernel(float *C, long long M, long long N, long long ldc,
                               long long strideC, long long batch, float beta,
                               const float *bias, int act) {
    const long long nrows = M * batch;
    const bool fused = bias != nullptr || act != sg::kActNone;
    for (long long gr = blockIdx.y; gr < nrows; gr += gridDim.y) {
        const long long b = gr / M, r = gr - b * M;
        float *row = C + b * strideC + r * ldc;
        for (long long c = blockIdx.x * static_cast<long long>(blockDim.x) + threadIdx.x; c < N;
             c += static_cast<long long>(gridDim.x) * blockDim.x) {
            if (fused)
                row[c] = sg::epilogue_value(0.0f, 0.0f, beta, bias, static_cast<int>(c), act,
                                            row + c);
            else
                row[c] = beta == 0.0f ? 0.0f : beta * row[c];
        }
    }
}

struct Args {
    long long M, N, K;
    float alpha, beta;
    const float *A;
    long long lda, sA;
    const float *B;
    long long ldb, sB;
    float *C;
    long long ldc, sC;
    long long batch;
    bool ta = false, tb = false;  // A stored K x M, B stored N x K
    const float *bias = nullptr;  // fused epilogue
    int act = 0;
};

// Checks shared by every entry point. Returns SGEMM_OK when the arguments are valid.
sgemm_status_t validate(const Args &a) {
    if (a.M < 0 || a.N < 0 || a.K < 0) return fail(SGEMM_ERR_INVALID_VALUE, "M, N and K must be >= 0");
    if (a.batch < 0) return fail(SGEMM_ERR_INVALID_VALUE, "batch must be >= 0");
    const long long acols = a.ta ? a.M : a.K, bcols = a.tb ? a.K : a.N;
    if (a.lda < (acols > 1 ? acols : 1))
        return fail(SGEMM_ERR_INVALID_VALUE, a.ta ? "lda < max(1, M) (A transposed)" : "lda < max(1, K)");
    if (a.ldb < (bcols > 1 ? bcols : 1))
        return fail(SGEMM_ERR_INVALID_VALUE, a.tb ? "ldb < max(1, K) (B transposed)" : "ldb < max(1, N)");
    if (a.ldc < (a.N > 1 ? a.N : 1)) return fail(SGEMM_ERR_INVALID_VALUE, "ldc < max(1, N)");
    if (a.sA < 0 || a.sB < 0 || a.sC < 0)
        return fail(SGEMM_ERR_INVALID_VALUE, "batch strides must be >= 0");
    if (a.M == 0 || a.N == 0 || a.batch == 0) return SGEMM_OK;
    if (a.batch > 1 && a.sC < a.M * a.ldc)
        return fail(SGEMM_ERR_INVALID_VALUE, "strideC < M * ldc: batch outputs would overlap");
    if (!a.C) return fail(SGEMM_ERR_INVALID_VALUE, "C is NULL");
    const bool reads_ab = a.alpha != 0.0f && a.K > 0;
    if (reads_ab && (!a.A || !a.B)) return fail(SGEMM_ERR_INVALID_VALUE, "A or B is NULL");
    return SGEMM_OK;
}

bool is_noop(const Args &a) { return a.M == 0 || a.N == 0 || a.batch == 0; }

sgemm_status_t check_limits(const Args &a) {
    if (a.M > kMaxDim || a.N > kMaxDim || a.K > kMaxDim || a.batch > kMaxDim)
        return fail(SGEMM_ERR_UNSUPPORTED, "a dimension exceeds 2^31 - 1");
    return SGEMM_OK;
}

sgemm_status_t run_scale(const Args &a, cudaStream_t stream) {
    const long long nrows = a.M * a.batch;
    const dim3 grid(static_cast<unsigned>((a.N + 255) / 256 < 8 ? (a.N + 255) / 256 : 8),
                    static_cast<unsigned>(nrows < 65535 ? nrows : 65535));
    scale_c_kernel<<<grid, 256, 0, stream>>>(a.C, a.M, a.N, a.ldc, a.sC, a.batch, a.beta, a.bias,
                                             a.act);
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return fail_cuda("scale kernel launch", err);
    return SGEMM_OK;
}

sg::SimtProblem to_problem(const Args &a) {
    sg::SimtProblem p;
    p.M = static_cast<int>(a.M);
    p.N = static_cast<int>(a.N);
    p.K = static_cast<int>(a.K);
    p.alpha = a.alpha;
    p.beta = a.beta;
    p.A = a.A;
    p.B = a.B;
    p.C = a.C;
    p.lda = a.lda;
    p.ldb = a.ldb;
    p.ldc = a.ldc;
    p.strideA = a.batch > 1 ? a.sA : 0;
    p.strideB = a.batch > 1 ? a.sB : 0;
    p.strideC = a.batch > 1 ? a.sC : 0;
    p.batch = static_cast<int>(a.batch);
    p.transA = a.ta;
    p.transB = a.tb;
    p.bias = a.bias;
    p.act = a.act;
    return p;
}

int choose_simt(const sg::SimtProblem &p) {
    const int forced = forced_config();
    if (forced >= 0 && sg::simt_config_supports(forced, p)) return forced;
    return sg::table_choose(p, sg::simt_device_sms());
}

sgemm_status_t run_simt(const Args &a, cudaStream_t stream) {
    sg::SimtProblem p = to_problem(a);
    if (p.transA || p.transB) {  // the tile kernels read op(A), op(B) row-major
        const char *detail = "";
        sg::SimtProblem q;
        cudaError_t err = sg::simt_untranspose(p, stream, &q, &detail);
        if (err != cudaSuccess) return fail_cuda(detail, err);
        p = q;
    }
    const int id = choose_simt(p);
    if (log_enabled())
        std::fprintf(stderr, "[sgemm] M=%lld N=%lld K=%lld batch=%lld -> %s\n", a.M, a.N, a.K,
                     a.batch, sg::simt_config(id).name);
    const char *detail = "";
    cudaError_t err = sg::simt_launch(id, p, stream, &detail);
    if (err != cudaSuccess) return fail_cuda(detail, err);
    return SGEMM_OK;
}

enum Path { kPathSimt, kPathTf32x3, kPathTf32 };

sgemm_status_t run_tensor(const Args &a, cudaStream_t stream, Path path) {
    const sg::SimtProblem p = to_problem(a);
    if (!sg::tf32x3_supports(p))
        return fail(SGEMM_ERR_UNSUPPORTED, "the TF32 paths take at most 65535 batch entries");
    const char *detail = "";
    cudaError_t err = path == kPathTf32 ? sg::tf32_launch(p, stream, &detail)
                                        : sg::tf32x3_launch(p, stream, &detail);
    if (err != cudaSuccess) return fail_cuda(detail, err);
    return SGEMM_OK;
}

bool have_device() {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess;
}

sgemm_status_t dispatch(const Args &a, void *stream_ptr, Path path) {
    t_last_error[0] = '\0';
    sgemm_status_t st = validate(a);
    if (st != SGEMM_OK) return st;
    if (is_noop(a)) return SGEMM_OK;
    st = check_limits(a);
    if (st != SGEMM_OK) return st;
    if (!have_device()) return fail(SGEMM_ERR_UNSUPPORTED, "no CUDA device available");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (a.alpha == 0.0f || a.K == 0) return run_scale(a, stream);
    return path == kPathSimt ? run_simt(a, stream) : run_tensor(a, stream, path);
}

// Device product used by each chunk of the host-memory path (the SIMT path).
cudaError_t chunk_gemm(long long M, long long N, long long K, float alpha, const float *A,
                       long long lda, const float *B, long long ldb, float beta, float *C,
                       long long ldc, cudaStream_t stream, const char **detail) {
    Args a{M, N, K, alpha, beta, A, lda, 0, B, ldb, 0, C, ldc, 0, 1};
    const sgemm_status_t st = (alpha == 0.0f || K == 0) ? run_scale(a, stream) : run_simt(a, stream);
    if (st != SGEMM_OK) {
        *detail = "a chunk's device product failed";
        return cudaErrorLaunchFailure;
    }
    return cudaSuccess;
}

// ---- layer operators on 16-bit values -----------------------------------------------------------

bool known_dtype(sgemm_dtype_t d) { return d == SGEMM_DTYPE_BF16 || d == SGEMM_DTYPE_F16; }
bool known_op(sgemm_op_t op) { return op == SGEMM_OP_N || op == SGEMM_OP_T; }
bool known_act(sgemm_activation_t a) { return a >= SGEMM_ACT_NONE && a <= SGEMM_ACT_SILU; }
bool short_ld(long long ld, long long cols) { return ld < (cols > 1 ? cols : 1); }
bool odd(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 1u) != 0; }
const uint16_t *in16(const void *p) { return static_cast<const uint16_t *>(p); }
uint16_t *out16(void *p) { return static_cast<uint16_t *>(p); }

sgemm_status_t check_linear(sgemm_dtype_t dtype, sgemm_op_t transw, sgemm_activation_t act,
                            int64_t M, int64_t N, int64_t K) {
    if (!known_dtype(dtype)) return fail(SGEMM_ERR_INVALID_VALUE, "unknown dtype");
    if (!known_op(transw))
        return fail(SGEMM_ERR_INVALID_VALUE, "transw must be SGEMM_OP_N or SGEMM_OP_T");
    if (!known_act(act)) return fail(SGEMM_ERR_INVALID_VALUE, "unknown activation");
    if (M < 0 || N < 0 || K < 0) return fail(SGEMM_ERR_INVALID_VALUE, "M, N and K must be >= 0");
    return SGEMM_OK;
}

sgemm_status_t check_layer_limits(int64_t M, int64_t N, int64_t K) {
    if (M > kMaxDim || N > kMaxDim || K > kMaxDim)
        return fail(SGEMM_ERR_UNSUPPORTED, "a dimension exceeds 2^31 - 1");
    if (!have_device()) return fail(SGEMM_ERR_UNSUPPORTED, "no CUDA device available");
    return SGEMM_OK;
}

const uint64_t kStandIn = 0;  // an aligned address

// The two arrays of an 8-bit checkpoint.
struct Codes8 {
    const int8_t *Q;
    int64_t ldq;
    const float *S;
    int64_t lds;
};

sgemm_status_t check_dtype(sgemm_dtype_t dtype) {
    return dtype == SGEMM_DTYPE_BF16 || dtype == SGEMM_DTYPE_F16 ? SGEMM_OK
                                                                 : fail(SGEMM_ERR_INVALID_VALUE, "unknown dtype");
}

// Of an M x N matrix, M and N >= 0.
sgemm_status_t check_codes(const Codes8 &c, int64_t M, int64_t N) {
    if (short_ld(c.ldq, N)) return fail(SGEMM_ERR_INVALID_VALUE, "a checkpoint's ldq < max(1, columns)");
    if (short_ld(c.lds, N / 64 + (N % 64 != 0)))
        return fail(SGEMM_ERR_INVALID_VALUE, "a checkpoint's lds < max(1, ceil(columns / 64))");
    if (M > 0 && N > 0 && (!c.Q || !c.S)) return fail(SGEMM_ERR_INVALID_VALUE, "a checkpoint's Q or S is NULL");
    if (reinterpret_cast<uintptr_t>(c.S) & 3u)
        return fail(SGEMM_ERR_INVALID_VALUE, "a checkpoint's S is not aligned to its type");
    return SGEMM_OK;
}

sg::Checkpoint8 to_checkpoint(const Codes8 &c, sgemm_dtype_t dtype, int64_t M, int64_t N) {
    sg::Checkpoint8 q;
    q.dtype = dtype;
    q.M = static_cast<int>(M);
    q.N = static_cast<int>(N);
    q.Q = const_cast<int8_t *>(c.Q);
    q.ldq = c.ldq;
    q.S = const_cast<float *>(c.S);
    q.lds = c.lds;
    return q;
}

sgemm_status_t checkpoint8(sgemm_dtype_t dtype, int64_t M, int64_t N, const void *X, int64_t ldx, const Codes8 &c,
                           bool save, cudaStream_t stream) {
    sgemm_status_t st = check_dtype(dtype);
    if (st != SGEMM_OK) return st;
    if (M < 0 || N < 0) return fail(SGEMM_ERR_INVALID_VALUE, "M and N must be >= 0");
    if (short_ld(ldx, N)) return fail(SGEMM_ERR_INVALID_VALUE, "ldx < max(1, N)");
    st = check_codes(c, M, N);
    if (st != SGEMM_OK) return st;
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!X) return fail(SGEMM_ERR_INVALID_VALUE, "X is NULL");
    if (odd(X)) return fail(SGEMM_ERR_INVALID_VALUE, "X is not aligned to its 2-byte type");
    st = check_layer_limits(M, N, 0);
    if (st != SGEMM_OK) return st;
    sg::Checkpoint8 q = to_checkpoint(c, dtype, M, N);
    const char *detail = "";
    cudaError_t err;
    if (save) {
        q.X = in16(X);
        q.ldx = ldx;
        err = sg::save8_launch(q, stream, &detail);
    } else {
        const sg::Restore8 r{q.dtype, q.M, q.N, q.Q, q.ldq, q.S, q.lds, const_cast<uint16_t *>(in16(X)), ldx};
        err = sg::restore8_launch(r, stream, &detail);
    }
    return err == cudaSuccess ? SGEMM_OK : fail_cuda(detail, err);
}

sgemm_status_t linear(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N, int64_t K,
                      const void *X, int64_t ldx, const void *W, int64_t ldw, const void *bias,
                      sgemm_activation_t act, const void *R, int64_t ldr, void *Y, int64_t ldy,
                      void *Z, int64_t ldz, const Codes8 *saved, cudaStream_t stream) {
    sgemm_status_t st = check_linear(dtype, transw, act, M, N, K);
    if (st == SGEMM_OK && saved) st = check_codes(*saved, M, N);
    if (st != SGEMM_OK) return st;
    if (short_ld(ldx, K)) return fail(SGEMM_ERR_INVALID_VALUE, "ldx < max(1, K)");
    if (short_ld(ldw, transw == SGEMM_OP_T ? K : N))
        return fail(SGEMM_ERR_INVALID_VALUE, transw == SGEMM_OP_T ? "ldw < max(1, K) (W transposed)"
                                                                  : "ldw < max(1, N)");
    if (R && short_ld(ldr, N)) return fail(SGEMM_ERR_INVALID_VALUE, "ldr < max(1, N)");
    if (short_ld(ldy, N)) return fail(SGEMM_ERR_INVALID_VALUE, "ldy < max(1, N)");
    if (Z && short_ld(ldz, N)) return fail(SGEMM_ERR_INVALID_VALUE, "ldz < max(1, N)");
    if (M == 0 || N == 0) return SGEMM_OK;
    if (!Y) return fail(SGEMM_ERR_INVALID_VALUE, "Y is NULL");
    if (K > 0 && (!X || !W)) return fail(SGEMM_ERR_INVALID_VALUE, "X or W is NULL");
    if (odd(X) || odd(W) || odd(bias) || odd(R) || odd(Y) || odd(Z))
        return fail(SGEMM_ERR_INVALID_VALUE, "a pointer is not aligned to its 2-byte type");
    if (Y == Z) return fail(SGEMM_ERR_INVALID_VALUE, "Y and Z are the same matrix");
    if ((R == Y && ldr != ldy) || (Z && R == Z))
        return fail(SGEMM_ERR_INVALID_VALUE, "R overlaps an output other than as Y itself");
    st = check_layer_limits(M, N, K);
    if (st != SGEMM_OK) return st;
    sg::Gemm16 g;
    g.dtype = dtype;
    g.M = static_cast<int>(M);
    g.N = static_cast<int>(N);
    g.K = static_cast<int>(K);
    g.A = in16(X);
    g.lda = ldx;
    g.B = in16(W);
    g.ldb = ldw;
    g.b_mn = transw == SGEMM_OP_N;
    g.D = out16(Y);
    g.ldd = ldy;
    g.bias = in16(bias);
    g.act = act;
    g.res = in16(R);
    g.ldr = ldr;
    g.pre = out16(Z);
    g.ldz = ldz;
    const char *detail = "";
    cudaError_t err;
    if (saved)
        err = sg::gemm16_save8_launch(g, to_checkpoint(*saved, dtype, M, N), stream, &detail);
    else
        err = sg::gemm16_launch(&g, 1, stream, &detail);
    return err == cudaSuccess ? SGEMM_OK : fail_cuda(detail, err);
}

sgemm_status_t linear_backward(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N,
                               int64_t K, const void *dY, int64_t lddy, const void *Z, int64_t ldz,
                               sgemm_activation_t act, const void *X, int64_t ldx, const void *W,
                               int64_t ldw, void *dX, int64_t lddx, void *dW, int64_t lddw,
                               float *db, cudaStream_t stream, const Codes8 *z8 = nullptr, bool only_check = false) {
    sgemm_status_t st = check_linear(dtype, transw, act, M, N, K);
    if (st != SGEMM_OK) return st;
    const bool t = transw == SGEMM_OP_T;
    const int64_t wcols = t ? K : N;
    if (short_ld(lddy, N)) return fail(SGEMM_ERR_INVALID_VALUE, "lddy < max(1, N)");
    if (act != SGEMM_ACT_NONE && short_ld(ldz, N)) return fail(SGEMM_ERR_INVALID_VALUE, "ldz < max(1, N)");
    if (dW && short_ld(ldx, K)) return fail(SGEMM_ERR_INVALID_VALUE, "ldx < max(1, K)");
    if (dX && short_ld(ldw, wcols))
        return fail(SGEMM_ERR_INVALID_VALUE, t ? "ldw < max(1, K) (W transposed)" : "ldw < max(1, N)");
    if (dX && short_ld(lddx, K)) return fail(SGEMM_ERR_INVALID_VALUE, "lddx < max(1, K)");
    if (dW && short_ld(lddw, wcols))
        return fail(SGEMM_ERR_INVALID_VALUE, t ? "lddw < max(1, K) (W transposed)" : "lddw < max(1, N)");
    const bool want_dx = dX && M > 0 && K > 0, want_dw = dW && N > 0 && K > 0, want_db = db && N > 0;
    if (!want_dx && !want_dw && !want_db) return SGEMM_OK;
    const bool reads = M > 0 && N > 0;
    if (reads && !dY) return fail(SGEMM_ERR_INVALID_VALUE, "dY is NULL");
    if (reads && act != SGEMM_ACT_NONE && !Z)
        return fail(SGEMM_ERR_INVALID_VALUE, "Z is NULL (the activation's gradient needs it)");
    if (reads && want_dw && !X) return fail(SGEMM_ERR_INVALID_VALUE, "X is NULL (dW needs it)");
    if (reads && want_dx && !W) return fail(SGEMM_ERR_INVALID_VALUE, "W is NULL (dX needs it)");
    if (odd(dY) || odd(Z) || odd(X) || odd(W) || odd(dX) || odd(dW) ||
        (reinterpret_cast<uintptr_t>(db) & 3u))
        return fail(SGEMM_ERR_INVALID_VALUE, "a pointer is not aligned to its type");
    st = check_layer_limits(M, N, K);
    if (st != SGEMM_OK || only_check) return st;

    const char *detail = "";
    const uint16_t *dz = in16(dY);
    long long lddz = lddy;
    cudaError_t err = cudaSuccess;
    // The products read dz: dY * act'(Z), or an aligned copy of a dY that TMA cannot address.
    const bool make_dz = reads && (want_dx || want_dw) &&
                         (act != SGEMM_ACT_NONE || !sg::tma_rows(dY, lddy));
    if (want_db || make_dz) {
        sg::ActGrad a;
        a.dtype = dtype;
        a.M = static_cast<int>(M);
        a.N = static_cast<int>(N);
        a.dy = in16(dY);
        a.lddy = lddy;
        if (z8) {
            a.zq = z8->Q;
            a.ldzq = z8->ldq;
            a.zs = z8->S;
            a.ldzs = z8->lds;
        } else {
            a.z = in16(Z);
            a.ldz = ldz;
        }
        a.act = act;
        a.db = db;
        if (make_dz) {
            lddz = (N + 7) / 8 * 8;
            void *p = nullptr;
            err = sg::layer_scratch(sg::kScratchDz, stream, static_cast<size_t>(M) * lddz * 2, &p, &detail);
            if (err != cudaSuccess) return fail_cuda(detail, err);
            a.dz = static_cast<uint16_t *>(p);
            a.lddz = lddz;
            dz = a.dz;
        }
        err = sg::act_grad_launch(a, stream, &detail);
        if (err != cudaSuccess) return fail_cuda(detail, err);
    }
    sg::Gemm16 list[2];
    int n = 0;
    if (want_dx) {  // dX = dZ . op(W)^T: K of this product is N, op(W)^T is N x K
        sg::Gemm16 &g = list[n++];
        g.dtype = dtype;
        g.M = static_cast<int>(M);
        g.N = static_cast<int>(K);
        g.K = static_cast<int>(N);
        g.A = dz;
        g.lda = lddz;
        g.a_mn = false;
        g.B = in16(W);
        g.ldb = ldw;
        g.b_mn = t;  // W stored N x K: rows run along this product's K
        g.D = out16(dX);
        g.ldd = lddx;
    }
    if (want_dw) {  // dW = dZ^T . X (N x K) or X^T . dZ (K x N): K of this product is M
        sg::Gemm16 &g = list[n++];
        g.dtype = dtype;
        g.M = static_cast<int>(t ? N : K);
        g.N = static_cast<int>(t ? K : N);
        g.K = static_cast<int>(M);
        g.A = t ? dz : in16(X);
        g.lda = t ? lddz : ldx;
        g.a_mn = true;
        g.B = t ? in16(X) : dz;
        g.ldb = t ? ldx : lddz;
        g.b_mn = true;
        g.D = out16(dW);
        g.ldd = lddw;
    }
    if (n > 0) {
        err = sg::gemm16_launch(list, n, stream, &detail);
        if (err != cudaSuccess) return fail_cuda(detail, err);
    }
    return SGEMM_OK;
}

// A checkpoint restored to scratch: *out and *ld then name an aligned 16-bit matrix.
cudaError_t restore_to_scratch(const Codes8 &c, sgemm_dtype_t dtype, int64_t M, int64_t N, sg::LayerScratch use,
                               cudaStream_t stream, const void **out, int64_t *ld, const char **detail) {
    const sg::Checkpoint8 q = to_checkpoint(c, dtype, M, N);
    sg::Restore8 r{q.dtype, q.M, q.N, q.Q, q.ldq, q.S, q.lds, nullptr, (N + 7) / 8 * 8};
    void *p = nullptr;
    const cudaError_t err = sg::layer_scratch(use, stream, static_cast<size_t>(M) * r.ldx * 2, &p, detail);
    if (err != cudaSuccess) return err;
    r.X = static_cast<uint16_t *>(p);
    *out = p;
    *ld = r.ldx;
    return sg::restore8_launch(r, stream, detail);
}

sgemm_status_t linear_backward8(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N, int64_t K,
                                const void *dY, int64_t lddy, const Codes8 &z, sgemm_activation_t act,
                                const Codes8 &x, const void *W, int64_t ldw, void *dX, int64_t lddx, void *dW,
                                int64_t lddw, float *db, cudaStream_t stream) {
    sgemm_status_t st = check_linear(dtype, transw, act, M, N, K);
    const bool want_dx = dX && M > 0 && N > 0 && K > 0, want_dw = dW && N > 0 && K > 0;
    const bool use_z = act != SGEMM_ACT_NONE && (want_dx || want_dw || (db && N > 0)) && M > 0;
    const bool use_x = want_dw && M > 0;
    if (st == SGEMM_OK && act != SGEMM_ACT_NONE) st = check_codes(z, use_z ? M : 0, N);
    if (st == SGEMM_OK && dW) st = check_codes(x, use_x ? M : 0, K);
    if (st != SGEMM_OK) return st;
    // The checks of linear_backward on the rest, with nothing queued, come first: a stand-in for what
    // is restored.
    const void *X = x.Q ? &kStandIn : nullptr, *Z = z.Q ? &kStandIn : nullptr;
    int64_t ldx = std::max<int64_t>(1, K), ldz = std::max<int64_t>(1, N);
    st = linear_backward(dtype, transw, M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX, lddx, dW, lddw, db,
                         stream, nullptr, true);
    if (st != SGEMM_OK) return st;
    const char *detail = "";
    cudaError_t err = cudaSuccess;
    // The gradient pass reads aligned codes itself; the product needs X in 16 bits.
    const bool z_direct = use_z && (reinterpret_cast<uintptr_t>(z.Q) & 7u) == 0 && z.ldq % 8 == 0;
    if (use_x) err = restore_to_scratch(x, dtype, M, K, sg::kScratchRestoreX, stream, &X, &ldx, &detail);
    if (err == cudaSuccess && use_z && !z_direct)
        err = restore_to_scratch(z, dtype, M, N, sg::kScratchRestoreZ, stream, &Z, &ldz, &detail);
    if (err != cudaSuccess) return fail_cuda(detail, err);
    return linear_backward(dtype, transw, M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX, lddx, dW, lddw, db,
                           stream, z_direct ? &z : nullptr);
}

// Checks what the loss and its gradient share.
sgemm_status_t check_head(const sg::Head16 &h, sgemm_dtype_t dtype, sgemm_op_t transw, int64_t T, int64_t V,
                          int64_t D) {
    const sgemm_status_t st = check_dtype(dtype);
    if (st != SGEMM_OK) return st;
    if (transw != SGEMM_OP_N && transw != SGEMM_OP_T)
        return fail(SGEMM_ERR_INVALID_VALUE, "transw must be SGEMM_OP_N or SGEMM_OP_T");
    if (T < 0) return fail(SGEMM_ERR_INVALID_VALUE, "T must be >= 0");
    if (V < 1 || D < 1) return fail(SGEMM_ERR_INVALID_VALUE, "V and D must be >= 1");
    if (short_ld(h.ldx, D)) return fail(SGEMM_ERR_INVALID_VALUE, "ldx < D");
    if (short_ld(h.ldw, h.w_dv ? V : D)) return fail(SGEMM_ERR_INVALID_VALUE, h.w_dv ? "ldw < V" : "ldw < D (W transposed)");
    return SGEMM_OK;
}

sgemm_status_t check_head_pointers(const sg::Head16 &h) {
    if (!h.X || !h.W) return fail(SGEMM_ERR_INVALID_VALUE, "X or W is NULL");
    if (!h.labels) return fail(SGEMM_ERR_INVALID_VALUE, "labels is NULL");
    auto off = [](const void *p, unsigned mask) { return (reinterpret_cast<uintptr_t>(p) & mask) != 0; };
    if (odd(h.X) || odd(h.W) || odd(h.dX) || odd(h.dW) || off(h.labels, 7u) || off(h.loss, 3u) || off(h.lse, 3u) ||
        off(h.dloss, 3u) || off(h.lse_in, 3u))
        return fail(SGEMM_ERR_INVALID_VALUE, "a pointer is not aligned to its type");
    return SGEMM_OK;
}

sgemm_status_t head(sg::Head16 h, bool gradient, sgemm_dtype_t dtype, sgemm_op_t transw, int64_t T, int64_t V,
                    int64_t D, cudaStream_t stream) {
    h.w_dv = transw == SGEMM_OP_N;
    sgemm_status_t st = check_head(h, dtype, transw, T, V, D);
    if (st != SGEMM_OK) return st;
    if (gradient) {
        if (h.incd < 0) return fail(SGEMM_ERR_INVALID_VALUE, "incd must be >= 0");
        if (h.dX && short_ld(h.lddx, D)) return fail(SGEMM_ERR_INVALID_VALUE, "lddx < D");
        if (h.dW && short_ld(h.lddw, h.w_dv ? V : D))
            return fail(SGEMM_ERR_INVALID_VALUE, h.w_dv ? "lddw < V" : "lddw < D (W transposed)");
        if (!h.dX && !h.dW) return SGEMM_OK;
        if (T == 0 && !h.dW) return SGEMM_OK;
    } else if (T == 0 || (!h.loss && !h.lse)) {
        return SGEMM_OK;
    }
    if (T > 0) {
        st = check_head_pointers(h);
        if (st != SGEMM_OK) return st;
        if (gradient && (!h.dloss || !h.lse_in)) return fail(SGEMM_ERR_INVALID_VALUE, "dloss or lse is NULL");
        if (h.loss && h.loss == h.lse) return fail(SGEMM_ERR_INVALID_VALUE, "loss and lse are the same array");
    } else if (odd(h.dW)) {
        return fail(SGEMM_ERR_INVALID_VALUE, "a pointer is not aligned to its type");
    }
    st = check_layer_limits(T, V, D);
    if (st != SGEMM_OK) return st;
    h.dtype = static_cast<int>(dtype);
    h.T = static_cast<int>(T);
    h.V = static_cast<int>(V);
    h.D = static_cast<int>(D);
    const char *detail = "";
    cudaError_t err;
    if (T == 0) {  // a gradient without tokens: a product over no k writes zeros
        sg::Gemm16 g;
        g.dtype = h.dtype;
        g.M = h.w_dv ? h.D : h.V;
        g.N = h.w_dv ? h.V : h.D;
        g.D = h.dW;
        g.ldd = h.lddw;
        err = sg::gemm16_launch(&g, 1, stream, &detail);
    } else {
        err = gradient ? sg::head16_grad_launch(h, stream, &detail) : sg::head16_launch(h, stream, &detail);
    }
    return err == cudaSuccess ? SGEMM_OK : fail_cuda(detail, err);
}

sgemm_status_t moe(const sg::Moe16 &m, int64_t T, int64_t E, int64_t topk, int64_t D, int64_t F,
                   cudaStream_t stream) {
    if (m.dtype != SGEMM_DTYPE_BF16 && m.dtype != SGEMM_DTYPE_F16)
        return fail(SGEMM_ERR_INVALID_VALUE, "unknown dtype");
    if (m.act < SGEMM_ACT_NONE || m.act > SGEMM_ACT_SILU)
        return fail(SGEMM_ERR_INVALID_VALUE, "unknown activation");
    if (T < 0 || D < 0 || F < 0) return fail(SGEMM_ERR_INVALID_VALUE, "T, D and F must be >= 0");
    if (E < 1) return fail(SGEMM_ERR_INVALID_VALUE, "E must be >= 1");
    if (topk < 1 || topk > E) return fail(SGEMM_ERR_INVALID_VALUE, "topk must be between 1 and E");
    if (short_ld(m.ldx, D)) return fail(SGEMM_ERR_INVALID_VALUE, "ldx < max(1, D)");
    if (short_ld(m.ldr, D)) return fail(SGEMM_ERR_INVALID_VALUE, "ldwr < max(1, D)");
    if (short_ld(m.ldu, D)) return fail(SGEMM_ERR_INVALID_VALUE, "ldu < max(1, D)");
    if (short_ld(m.ldd, F)) return fail(SGEMM_ERR_INVALID_VALUE, "ldd < max(1, F)");
    if (m.su < 0 || m.sd < 0 || (E > 1 && (F > m.su / m.ldu || D > m.sd / m.ldd)))
        return fail(SGEMM_ERR_INVALID_VALUE, "strideu < F * ldu or strided < D * ldd");
    if (m.R && short_ld(m.ldres, D)) return fail(SGEMM_ERR_INVALID_VALUE, "ldr < max(1, D)");
    if (short_ld(m.ldy, D)) return fail(SGEMM_ERR_INVALID_VALUE, "ldy < max(1, D)");
    if (T > sg::kMoeMaxTokens || E > sg::kMoeMaxExperts || topk > sg::kMoeMaxTopk)
        return fail(SGEMM_ERR_UNSUPPORTED, "sgemm_moe takes at most 64 tokens, 512 experts and topk 16");
    if (T == 0) return SGEMM_OK;
    if (D > 0 && !m.Y) return fail(SGEMM_ERR_INVALID_VALUE, "Y is NULL");
    if (D > 0 && (!m.X || !m.Wr)) return fail(SGEMM_ERR_INVALID_VALUE, "X or Wr is NULL");
    if (D > 0 && F > 0 && (!m.Wu || !m.Wd)) return fail(SGEMM_ERR_INVALID_VALUE, "Wup or Wdown is NULL");
    if (odd(m.X) || odd(m.Wr) || odd(m.Wg) || odd(m.Wu) || odd(m.Wd) || odd(m.R) || odd(m.Y) ||
        (reinterpret_cast<uintptr_t>(m.index) & 3u) || (reinterpret_cast<uintptr_t>(m.weight) & 3u))
        return fail(SGEMM_ERR_INVALID_VALUE, "a pointer is not aligned to its type");
    if (m.R && m.R == m.Y && m.ldres != m.ldy)
        return fail(SGEMM_ERR_INVALID_VALUE, "R overlaps Y other than as Y itself");
    const sgemm_status_t st = check_layer_limits(D, F, 0);
    if (st != SGEMM_OK) return st;
    sg::Moe16 q = m;
    q.T = static_cast<int>(T);
    q.E = static_cast<int>(E);
    q.k = static_cast<int>(topk);
    q.D = static_cast<int>(D);
    q.F = static_cast<int>(F);
    const char *detail = "";
    const cudaError_t err = sg::moe16_launch(q, stream, &detail);
    return err == cudaSuccess ? SGEMM_OK : fail_cuda(detail, err);
}

// The launches of one layer operator's call share the stream's scratch, and a larger call moves it:
// calls from several host threads, of the same operator or not, queue theirs one call at a time.
// Freeing or clearing the scratch takes the same lock.
std::mutex g_layer_queueing;

// Runs `body` under that lock, turning a C++ exception (host memory exhausted) into a status.
template <typename Body>
sgemm_status_t guarded(Body body) {
    t_last_error[0] = '\0';
    try {
        std::lock_guard<std::mutex> lock(g_layer_queueing);
        return body();
    } catch (...) {
        return fail(SGEMM_ERR_LAUNCH, "out of host memory");
    }
}

}  // namespace

extern "C" {

sgemm_status_t sgemm_linear(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N,
                            int64_t K, const void *X, int64_t ldx, const void *W, int64_t ldw,
                            const void *bias, sgemm_activation_t act, const void *R, int64_t ldr,
                            void *Y, int64_t ldy, void *Z, int64_t ldz, void *stream) {
    return guarded([&] {
        return linear(dtype, transw, M, N, K, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, Z, ldz,
                      nullptr, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_linear_backward(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N,
                                     int64_t K, const void *dY, int64_t lddy, const void *Z,
                                     int64_t ldz, sgemm_activation_t act, const void *X,
                                     int64_t ldx, const void *W, int64_t ldw, void *dX,
                                     int64_t lddx, void *dW, int64_t lddw, float *db,
                                     void *stream) {
    return guarded([&] {
        return linear_backward(dtype, transw, M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX,
                               lddx, dW, lddw, db, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_checkpoint8(sgemm_dtype_t dtype, int64_t M, int64_t N, const void *X, int64_t ldx, int8_t *Q,
                                 int64_t ldq, float *S, int64_t lds, void *stream) {
    return guarded([&] {
        return checkpoint8(dtype, M, N, X, ldx, {Q, ldq, S, lds}, true, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_restore8(sgemm_dtype_t dtype, int64_t M, int64_t N, const int8_t *Q, int64_t ldq, const float *S,
                              int64_t lds, void *X, int64_t ldx, void *stream) {
    return guarded([&] {
        return checkpoint8(dtype, M, N, X, ldx, {Q, ldq, S, lds}, false, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_linear_checkpoint8(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N, int64_t K,
                                        const void *X, int64_t ldx, const void *W, int64_t ldw, const void *bias,
                                        sgemm_activation_t act, const void *R, int64_t ldr, void *Y, int64_t ldy,
                                        int8_t *Zq, int64_t ldzq, float *Zs, int64_t ldzs, void *stream) {
    return guarded([&] {
        const Codes8 saved{Zq, ldzq, Zs, ldzs};
        return linear(dtype, transw, M, N, K, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, nullptr, 0, &saved,
                      static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_linear_backward_checkpoint8(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t M, int64_t N,
                                                 int64_t K, const void *dY, int64_t lddy, const int8_t *Zq,
                                                 int64_t ldzq, const float *Zs, int64_t ldzs, sgemm_activation_t act,
                                                 const int8_t *Xq, int64_t ldxq, const float *Xs, int64_t ldxs,
                                                 const void *W, int64_t ldw, void *dX, int64_t lddx, void *dW,
                                                 int64_t lddw, float *db, void *stream) {
    return guarded([&] {
        return linear_backward8(dtype, transw, M, N, K, dY, lddy, {Zq, ldzq, Zs, ldzs}, act, {Xq, ldxq, Xs, ldxs}, W,
                                ldw, dX, lddx, dW, lddw, db, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_cross_entropy(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t T, int64_t V, int64_t D,
                                   const void *X, int64_t ldx, const void *W, int64_t ldw, const int64_t *labels,
                                   float *loss, float *lse, void *stream) {
    return guarded([&] {
        sg::Head16 h;
        h.X = in16(X);
        h.ldx = ldx;
        h.W = in16(W);
        h.ldw = ldw;
        h.labels = labels;
        h.loss = loss;
        h.lse = lse;
        return head(h, false, dtype, transw, T, V, D, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_cross_entropy_backward(sgemm_dtype_t dtype, sgemm_op_t transw, int64_t T, int64_t V, int64_t D,
                                            const float *dloss, int64_t incd, const void *X, int64_t ldx,
                                            const void *W, int64_t ldw, const int64_t *labels, const float *lse,
                                            void *dX, int64_t lddx, void *dW, int64_t lddw, void *stream) {
    return guarded([&] {
        sg::Head16 h;
        h.X = in16(X);
        h.ldx = ldx;
        h.W = in16(W);
        h.ldw = ldw;
        h.labels = labels;
        h.dloss = dloss;
        h.incd = incd;
        h.lse_in = lse;
        h.dX = out16(dX);
        h.lddx = lddx;
        h.dW = out16(dW);
        h.lddw = lddw;
        return head(h, true, dtype, transw, T, V, D, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm_moe(sgemm_dtype_t dtype, sgemm_activation_t act, int64_t T, int64_t E,
                         int64_t topk, int64_t D, int64_t F, const void *X, int64_t ldx,
                         const void *Wr, int64_t ldwr, const void *Wgate, const void *Wup,
                         int64_t ldu, int64_t strideu, const void *Wdown, int64_t ldd,
                         int64_t strided, int renormalize, const uint8_t *active, const void *R,
                         int64_t ldr, void *Y, int64_t ldy, int32_t *topk_index,
                         float *topk_weight, void *stream) {
    return guarded([&] {
        sg::Moe16 m;
        m.dtype = static_cast<int>(dtype);
        m.act = static_cast<int>(act);
        m.X = in16(X);
        m.ldx = ldx;
        m.Wr = in16(Wr);
        m.ldr = ldwr;
        m.Wg = in16(Wgate);
        m.Wu = in16(Wup);
        m.ldu = ldu;
        m.su = strideu;
        m.Wd = in16(Wdown);
        m.ldd = ldd;
        m.sd = strided;
        m.renormalize = renormalize != 0;
        m.active = active;
        m.R = in16(R);
        m.ldres = ldr;
        m.Y = out16(Y);
        m.ldy = ldy;
        m.index = topk_index;
        m.weight = topk_weight;
        return moe(m, T, E, topk, D, F, static_cast<cudaStream_t>(stream));
    });
}

sgemm_status_t sgemm(int64_t M, int64_t N, int64_t K, float alpha, const float *A, int64_t lda,
                     const float *B, int64_t ldb, float beta, float *C, int64_t ldc,
                     void *stream) {
    Args a{M, N, K, alpha, beta, A, lda, 0, B, ldb, 0, C, ldc, 0, 1};
    return dispatch(a, stream, kPathSimt);
}

sgemm_status_t sgemm_strided_batched(int64_t M, int64_t N, int64_t K, float alpha,
                                     const float *A, int64_t lda, int64_t strideA,
                                     const float *B, int64_t ldb, int64_t strideB, float beta,
                                     float *C, int64_t ldc, int64_t strideC, int64_t batch,
                                     void *stream) {
    Args a{M, N, K, alpha, beta, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch};
    return dispatch(a, stream, kPathSimt);
}

sgemm_status_t sgemm_3xtf32(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                            int64_t lda, const float *B, int64_t ldb, float beta, float *C,
                            int64_t ldc, void *stream) {
    Args a{M, N, K, alpha, beta, A, lda, 0, B, ldb, 0, C, ldc, 0, 1};
    return dispatch(a, stream, kPathTf32x3);
}

sgemm_status_t sgemm_3xtf32_strided_batched(int64_t M, int64_t N, int64_t K, float alpha,
                                            const float *A, int64_t lda, int64_t strideA,
                                            const float *B, int64_t ldb, int64_t strideB,
                                            float beta, float *C, int64_t ldc, int64_t strideC,
                                            int64_t batch, void *stream) {
    Args a{M, N, K, alpha, beta, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch};
    return dispatch(a, stream, kPathTf32x3);
}

sgemm_status_t sgemm_tf32(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                          int64_t lda, const float *B, int64_t ldb, float beta, float *C,
                          int64_t ldc, void *stream) {
    Args a{M, N, K, alpha, beta, A, lda, 0, B, ldb, 0, C, ldc, 0, 1};
    return dispatch(a, stream, kPathTf32);
}

sgemm_status_t sgemm_tf32_strided_batched(int64_t M, int64_t N, int64_t K, float alpha,
                                          const float *A, int64_t lda, int64_t strideA,
                                          const float *B, int64_t ldb, int64_t strideB,
                                          float beta, float *C, int64_t ldc, int64_t strideC,
                                          int64_t batch, void *stream) {
    Args a{M, N, K, alpha, beta, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch};
    return dispatch(a, stream, kPathTf32);
}

sgemm_status_t sgemm_noalloc(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                             int64_t lda, const float *B, int64_t ldb, float beta, float *C,
                             int64_t ldc, void *stream_ptr) {
    Args a{M, N, K, alpha, beta, A, lda, 0, B, ldb, 0, C, ldc, 0, 1};
    t_last_error[0] = '\0';
    sgemm_status_t st = validate(a);
    if (st != SGEMM_OK) return st;
    if (is_noop(a)) return SGEMM_OK;
    st = check_limits(a);
    if (st != SGEMM_OK) return st;
    if (!have_device()) return fail(SGEMM_ERR_UNSUPPORTED, "no CUDA device available");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    if (a.alpha == 0.0f || a.K == 0) return run_scale(a, stream);  // allocates nothing either
    const char *detail = "";
    cudaError_t err = sg::simt_launch_noalloc(to_problem(a), stream, &detail);
    if (err == cudaErrorNotSupported) return fail(SGEMM_ERR_UNSUPPORTED, detail);
    if (err != cudaSuccess) return fail_cuda(detail, err);
    return SGEMM_OK;
}

sgemm_status_t sgemm_selftest_bounded_wait(int which, void *stream_ptr) {
    t_last_error[0] = '\0';
    if (which != 0 && which != 1) return fail(SGEMM_ERR_INVALID_VALUE, "which must be 0 or 1");
    if (!have_device()) return fail(SGEMM_ERR_UNSUPPORTED, "no CUDA device available");
    cudaError_t err = sg::simt_selftest_wait(which, static_cast<cudaStream_t>(stream_ptr));
    if (err != cudaSuccess) return fail_cuda("self-test kernel launch", err);
    return SGEMM_OK;
}

sgemm_status_t sgemm_fused_strided_batched(sgemm_op_t transa, sgemm_op_t transb,
                                           sgemm_path_t path, int64_t M, int64_t N, int64_t K,
                                           float alpha, const float *A, int64_t lda,
                                           int64_t strideA, const float *B, int64_t ldb,
                                           int64_t strideB, float beta, float *C, int64_t ldc,
                                           int64_t strideC, int64_t batch, const float *bias,
                                           sgemm_activation_t act, void *stream) {
    t_last_error[0] = '\0';
    if (act < SGEMM_ACT_NONE || act > SGEMM_ACT_SILU)
        return fail(SGEMM_ERR_INVALID_VALUE, "unknown activation");
    if ((transa != SGEMM_OP_N && transa != SGEMM_OP_T) ||
        (transb != SGEMM_OP_N && transb != SGEMM_OP_T))
        return fail(SGEMM_ERR_INVALID_VALUE, "transa and transb must be SGEMM_OP_N or SGEMM_OP_T");
    Path pth;
    switch (path) {
        case SGEMM_PATH_SIMT: pth = kPathSimt; break;
        case SGEMM_PATH_3XTF32: pth = kPathTf32x3; break;
        case SGEMM_PATH_TF32: pth = kPathTf32; break;
        default: return fail(SGEMM_ERR_INVALID_VALUE, "unknown path");
    }
    Args a{M, N, K, alpha, beta, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch};
    a.ta = transa == SGEMM_OP_T;
    a.tb = transb == SGEMM_OP_T;
    a.bias = bias;
    a.act = static_cast<int>(act);
    return dispatch(a, stream, pth);
}

sgemm_status_t sgemm_fused(sgemm_op_t transa, sgemm_op_t transb, sgemm_path_t path, int64_t M,
                           int64_t N, int64_t K, float alpha, const float *A, int64_t lda,
                           const float *B, int64_t ldb, float beta, float *C, int64_t ldc,
                           const float *bias, sgemm_activation_t act, void *stream) {
    return sgemm_fused_strided_batched(transa, transb, path, M, N, K, alpha, A, lda, 0, B, ldb, 0,
                                       beta, C, ldc, 0, 1, bias, act, stream);
}

sgemm_status_t sgemm_ex_strided_batched(sgemm_op_t transa, sgemm_op_t transb, sgemm_path_t path,
                                        int64_t M, int64_t N, int64_t K, float alpha,
                                        const float *A, int64_t lda, int64_t strideA,
                                        const float *B, int64_t ldb, int64_t strideB, float beta,
                                        float *C, int64_t ldc, int64_t strideC, int64_t batch,
                                        void *stream) {
    t_last_error[0] = '\0';
    if ((transa != SGEMM_OP_N && transa != SGEMM_OP_T) ||
        (transb != SGEMM_OP_N && transb != SGEMM_OP_T))
        return fail(SGEMM_ERR_INVALID_VALUE, "transa and transb must be SGEMM_OP_N or SGEMM_OP_T");
    Path pth;
    switch (path) {
        case SGEMM_PATH_SIMT: pth = kPathSimt; break;
        case SGEMM_PATH_3XTF32: pth = kPathTf32x3; break;
        case SGEMM_PATH_TF32: pth = kPathTf32; break;
        default: return fail(SGEMM_ERR_INVALID_VALUE, "unknown path");
    }
    Args a{M, N, K, alpha, beta, A, lda, strideA, B, ldb, strideB, C, ldc, strideC, batch};
    a.ta = transa == SGEMM_OP_T;
    a.tb = transb == SGEMM_OP_T;
    return dispatch(a, stream, pth);
}

sgemm_status_t sgemm_ex(sgemm_op_t transa, sgemm_op_t transb, sgemm_path_t path, int64_t M,
                        int64_t N, int64_t K, float alpha, const float *A, int64_t lda,
                        const float *B, int64_t ldb, float beta, float *C, int64_t ldc,
                        void *stream) {
    return sgemm_ex_strided_batched(transa, transb, path, M, N, K, alpha, A, lda, 0, B, ldb, 0,
                                    beta, C, ldc, 0, 1, stream);
}

sgemm_status_t sgemm_host(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                          int64_t lda, const float *B, int64_t ldb, float beta, float *C,
                          int64_t ldc, void *stream_ptr) {
    Args a{M, N, K, alpha, beta, A, lda, 0, B, ldb, 0, C, ldc, 0, 1};
    t_last_error[0] = '\0';
    sgemm_status_t st = validate(a);
    if (st != SGEMM_OK) return st;
    if (is_noop(a)) return SGEMM_OK;
    st = check_limits(a);
    if (st != SGEMM_OK) return st;
    if (!have_device()) return fail(SGEMM_ERR_UNSUPPORTED, "no CUDA device available");
    const sg::HostProblem hp{M, N, K, alpha, beta, A, lda, B, ldb, C, ldc};
    const char *detail = "";
    cudaError_t err = sg::host_gemm(hp, static_cast<cudaStream_t>(stream_ptr), chunk_gemm, &detail);
    if (err != cudaSuccess) {
        if (t_last_error[0] != '\0') return SGEMM_ERR_LAUNCH;  // the chunk's own message stands
        return fail_cuda(detail, err);
    }
    return SGEMM_OK;
}

const char *sgemm_status_string(sgemm_status_t status) {
    switch (status) {
        case SGEMM_OK: return "SGEMM_OK";
        case SGEMM_ERR_INVALID_VALUE: return "SGEMM_ERR_INVALID_VALUE";
        case SGEMM_ERR_LAUNCH: return "SGEMM_ERR_LAUNCH";
        case SGEMM_ERR_TIMEOUT: return "SGEMM_ERR_TIMEOUT";
        case SGEMM_ERR_UNSUPPORTED: return "SGEMM_ERR_UNSUPPORTED";
    }
    return "SGEMM_(unknown status)";
}

const char *sgemm_last_error(void) { return t_last_error; }

sgemm_status_t sgemm_device_status(void *stream_ptr) {
    t_last_error[0] = '\0';
    if (!have_device()) return fail(SGEMM_ERR_UNSUPPORTED, "no CUDA device available");
    cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    cudaError_t err = cudaStreamSynchronize(stream);
    if (err != cudaSuccess) return fail_cuda("stream synchronize", err);
    const unsigned int word = sg::take_fault_words(stream);
    if (word & sg::kFaultTimeout) {
        std::lock_guard<std::mutex> lock(g_layer_queueing);
        sg::layer_scratch_distrust();
        return fail(SGEMM_ERR_TIMEOUT, "a bounded wait inside a kernel expired");
    }
    return SGEMM_OK;
}

sgemm_status_t sgemm_release_workspace(void) {
    t_last_error[0] = '\0';
    if (!have_device()) return SGEMM_OK;
    cudaError_t err = cudaDeviceSynchronize();
    if (err != cudaSuccess) return fail_cuda("device synchronize", err);
    err = sg::release_workspaces();
    cudaError_t err3 = sg::release_pack_workspaces();
    cudaError_t err4 = sg::release_host_buffers();
    if (err3 == cudaSuccess) err3 = err4;
    {
        // A call that another thread has queued since the synchronisation above may use the buffers.
        std::lock_guard<std::mutex> lock(g_layer_queueing);
        cudaError_t err5 = cudaDeviceSynchronize();
        if (err5 == cudaSuccess) err5 = sg::release_layer_workspaces();
        if (err3 == cudaSuccess) err3 = err5;
    }
    cudaError_t err2 = sg::tf32x3_release_workspaces();
    if (err == cudaSuccess) err = err3;
    if (err != cudaSuccess) return fail_cuda("workspace free", err);
    if (err2 != cudaSuccess) return fail_cuda("split workspace free", err2);
    return SGEMM_OK;
}

int sgemm_num_configs(void) { return sg::simt_num_configs(); }

const char *sgemm_config_name(int id) {
    if (id < 0 || id >= sg::simt_num_configs()) return nullptr;
    return sg::simt_config(id).name;
}

int sgemm_select_config(int64_t M, int64_t N, int64_t K, float alpha, const float *A,
                        int64_t lda, const float *B, int64_t ldb, const float *C, int64_t ldc,
                        int64_t batch) {
    Args a{M, N, K, alpha, 0.0f, A, lda, 0, B, ldb, 0, const_cast<float *>(C), ldc, 0, batch};
    if (batch > 1) {
        a.sA = M * lda;
        a.sB = K * ldb;
        a.sC = M * ldc;
    }
    if (validate(a) != SGEMM_OK || is_noop(a) || check_limits(a) != SGEMM_OK) return -1;
    if (alpha == 0.0f || K == 0) return -1;
    return choose_simt(to_problem(a));
}

sgemm_status_t sgemm_force_config(int id) {
    if (id < -1 || id >= sg::simt_num_configs())
        return fail(SGEMM_ERR_INVALID_VALUE, "unknown configuration id");
    g_forced_config.store(id);
    return SGEMM_OK;
}

}  // extern "C"
