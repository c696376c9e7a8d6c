"""GB300 single-precision GEMM: Python binding of the C ABI declared in ``include/sgemm.h``.

This module only marshals arguments: every step of C = alpha * (A . B) + beta * C runs in
the CUDA kernels of ``libsgemm_gb300.so`` (built in-tree by ``_build.build()``). There is no
CPU fallback: if the library is missing, every call raises ``RuntimeError``.

Pointer arguments accept either an integer device address or a torch CUDA tensor (its
``data_ptr()`` is passed). ``stream`` is an integer ``cudaStream_t``, a ``torch.cuda.Stream``
or None (torch's current stream when torch has CUDA, else the legacy default stream).
Non-OK statuses raise ``SgemmError`` carrying the status code and the library's message.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

__all__ = [
    "SgemmError", "library_path", "lib", "sgemm", "sgemm_strided_batched", "sgemm_3xtf32",
    "sgemm_3xtf32_strided_batched", "sgemm_tf32", "sgemm_tf32_strided_batched", "sgemm_ex",
    "sgemm_ex_strided_batched", "sgemm_fused", "sgemm_fused_strided_batched", "sgemm_host",
    "sgemm_noalloc", "sgemm_status_string", "sgemm_last_error",
    "sgemm_device_status", "sgemm_release_workspace", "sgemm_num_configs",
    "sgemm_config_name", "sgemm_select_config", "sgemm_force_config",
    "sgemm_selftest_bounded_wait", "matmul",
    "sgemm_linear", "sgemm_linear_backward", "sgemm_moe", "linear", "linear_backward", "moe",
    "sgemm_checkpoint8", "sgemm_restore8", "sgemm_linear_checkpoint8",
    "sgemm_linear_backward_checkpoint8", "sgemm_cross_entropy", "sgemm_cross_entropy_backward",
    "Checkpoint8", "checkpoint8", "restore8", "cross_entropy", "cross_entropy_backward",
    "SGEMM_DTYPE_BF16", "SGEMM_DTYPE_F16",
    "SGEMM_OK", "SGEMM_ERR_INVALID_VALUE", "SGEMM_ERR_LAUNCH", "SGEMM_ERR_TIMEOUT",
    "SGEMM_ERR_UNSUPPORTED",
]

SGEMM_OK = 0
SGEMM_ERR_INVALID_VALUE = 1
SGEMM_ERR_LAUNCH = 2
SGEMM_ERR_TIMEOUT = 3
SGEMM_ERR_UNSUPPORTED = 4

SGEMM_OP_N, SGEMM_OP_T = 0, 1
SGEMM_PATH_SIMT, SGEMM_PATH_3XTF32, SGEMM_PATH_TF32 = 0, 1, 2
_PATHS = {"simt": SGEMM_PATH_SIMT, "3xtf32": SGEMM_PATH_3XTF32, "tf32": SGEMM_PATH_TF32}
SGEMM_DTYPE_BF16, SGEMM_DTYPE_F16 = 0, 1
_DTYPES = {"torch.bfloat16": SGEMM_DTYPE_BF16, "torch.float16": SGEMM_DTYPE_F16,
           "bf16": SGEMM_DTYPE_BF16, "f16": SGEMM_DTYPE_F16}
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_LIBRARY = Path(__file__).resolve().with_name("libsgemm_gb300.so")
_lib = None


class SgemmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def library_path() -> Path:
    return _LIBRARY


def lib() -> ctypes.CDLL:
    """The loaded C library (raises RuntimeError when it has not been built)."""
    global _lib
    if _lib is None:
        if not _LIBRARY.exists():
            raise RuntimeError(f"{_LIBRARY.name} is not built; run "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        _lib = _bind(ctypes.CDLL(str(_LIBRARY)))
    return _lib


def _bind(L):
    i64, f32, p, i32 = ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_int
    gemm = [i64, i64, i64, f32, p, i64, p, i64, f32, p, i64, p]
    batched = [i64, i64, i64, f32, p, i64, i64, p, i64, i64, f32, p, i64, i64, i64, p]
    for name, args in (("sgemm", gemm), ("sgemm_3xtf32", gemm), ("sgemm_noalloc", gemm),
                       ("sgemm_host", gemm),
                       ("sgemm_tf32", gemm), ("sgemm_strided_batched", batched),
                       ("sgemm_3xtf32_strided_batched", batched),
                       ("sgemm_tf32_strided_batched", batched)):
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = i32
    L.sgemm_ex.argtypes = [i32, i32, i32] + gemm
    L.sgemm_ex.restype = i32
    L.sgemm_ex_strided_batched.argtypes = [i32, i32, i32] + batched
    L.sgemm_ex_strided_batched.restype = i32
    L.sgemm_fused.argtypes = [i32, i32, i32] + gemm[:-1] + [p, i32, p]
    L.sgemm_fused.restype = i32
    L.sgemm_fused_strided_batched.argtypes = [i32, i32, i32] + batched[:-1] + [p, i32, p]
    L.sgemm_fused_strided_batched.restype = i32
    L.sgemm_linear.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, i32, p, i64, p, i64,
                               p, i64, p]
    L.sgemm_linear.restype = i32
    L.sgemm_linear_backward.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, i32, p, i64, p,
                                        i64, p, i64, p, i64, p, p]
    L.sgemm_linear_backward.restype = i32
    L.sgemm_moe.argtypes = [i32, i32, i64, i64, i64, i64, i64, p, i64, p, i64, p, p, i64, i64, p,
                            i64, i64, i32, p, p, i64, p, i64, p, p, p]
    L.sgemm_moe.restype = i32
    L.sgemm_checkpoint8.argtypes = [i32, i64, i64, p, i64, p, i64, p, i64, p]
    L.sgemm_checkpoint8.restype = i32
    L.sgemm_restore8.argtypes = [i32, i64, i64, p, i64, p, i64, p, i64, p]
    L.sgemm_restore8.restype = i32
    L.sgemm_linear_checkpoint8.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, i32, p, i64, p,
                                           i64, p, i64, p, i64, p]
    L.sgemm_linear_checkpoint8.restype = i32
    L.sgemm_linear_backward_checkpoint8.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, i64,
                                                    i32, p, i64, p, i64, p, i64, p, i64, p, i64, p, p]
    L.sgemm_linear_backward_checkpoint8.restype = i32
    L.sgemm_cross_entropy.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, p, p, p]
    L.sgemm_cross_entropy.restype = i32
    L.sgemm_cross_entropy_backward.argtypes = [i32, i32, i64, i64, i64, p, i64, p, i64, p, i64, p, p,
                                               p, i64, p, i64, p]
    L.sgemm_cross_entropy_backward.restype = i32
    L.sgemm_status_string.argtypes = [i32]
    L.sgemm_status_string.restype = ctypes.c_char_p
    L.sgemm_last_error.argtypes = []
    L.sgemm_last_error.restype = ctypes.c_char_p
    L.sgemm_device_status.argtypes = [p]
    L.sgemm_device_status.restype = i32
    L.sgemm_release_workspace.argtypes = []
    L.sgemm_release_workspace.restype = i32
    L.sgemm_num_configs.argtypes = []
    L.sgemm_num_configs.restype = i32
    L.sgemm_config_name.argtypes = [i32]
    L.sgemm_config_name.restype = ctypes.c_char_p
    L.sgemm_select_config.argtypes = [i64, i64, i64, f32, p, i64, p, i64, p, i64, i64]
    L.sgemm_select_config.restype = i32
    L.sgemm_force_config.argtypes = [i32]
    L.sgemm_force_config.restype = i32
    L.sgemm_selftest_bounded_wait.argtypes = [i32, p]
    L.sgemm_selftest_bounded_wait.restype = i32
    return L


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    data_ptr = getattr(x, "data_ptr", None)
    if data_ptr is None:
        raise TypeError(f"expected a device address or a CUDA tensor, got {type(x).__name__}")
    if not x.is_cuda:
        raise TypeError("tensor arguments must live on a CUDA device")
    if str(x.dtype) != "torch.float32":
        raise TypeError("tensor arguments must be float32")
    return data_ptr()


def _stream(s):
    if s is None:
        try:
            import torch
            if torch.cuda.is_available():
                return torch.cuda.current_stream().cuda_stream
        except ImportError:
            pass
        return None
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(status: int) -> None:
    if status != SGEMM_OK:
        L = lib()
        msg = (L.sgemm_last_error() or b"").decode() or L.sgemm_status_string(status).decode()
        raise SgemmError(status, msg)


def sgemm(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C = alpha * (A . B) + beta * C on the FP32 SIMT path (asynchronous on ``stream``)."""
    _check(lib().sgemm(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, beta, _ptr(C), ldc,
                       _stream(stream)))


def sgemm_strided_batched(M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                          strideC, batch, stream=None) -> None:
    """``batch`` products; problem b uses A + b*strideA, B + b*strideB, C + b*strideC."""
    _check(lib().sgemm_strided_batched(M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb,
                                       strideB, beta, _ptr(C), ldc, strideC, batch,
                                       _stream(stream)))


def sgemm_3xtf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """The same operation on the tcgen05 tensor cores with the 3xTF32 split."""
    _check(lib().sgemm_3xtf32(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, beta, _ptr(C), ldc,
                              _stream(stream)))


def sgemm_3xtf32_strided_batched(M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C,
                                 ldc, strideC, batch, stream=None) -> None:
    _check(lib().sgemm_3xtf32_strided_batched(M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B),
                                              ldb, strideB, beta, _ptr(C), ldc, strideC, batch,
                                              _stream(stream)))


def sgemm_tf32(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """One TF32 product per multiply-add: faster, TF32 accuracy (see include/sgemm.h)."""
    _check(lib().sgemm_tf32(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, beta, _ptr(C), ldc,
                            _stream(stream)))


def sgemm_tf32_strided_batched(M, N, K, alpha, A, lda, strideA, B, ldb, strideB, beta, C, ldc,
                               strideC, batch, stream=None) -> None:
    _check(lib().sgemm_tf32_strided_batched(M, N, K, alpha, _ptr(A), lda, strideA, _ptr(B), ldb,
                                            strideB, beta, _ptr(C), ldc, strideC, batch,
                                            _stream(stream)))


def _op(t) -> int:
    if t in (0, 1):
        return int(t)
    if isinstance(t, str) and t.upper() in ("N", "T"):
        return SGEMM_OP_T if t.upper() == "T" else SGEMM_OP_N
    return int(bool(t))


def sgemm_ex(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, path="simt",
             stream=None) -> None:
    """C = alpha * op(A) op(B) + beta * C; transa / transb are 'N' / 'T' (or 0 / 1),
    path is 'simt', '3xtf32' or 'tf32' (or its enum value)."""
    pth = _PATHS.get(path, path) if isinstance(path, str) else int(path)
    _check(lib().sgemm_ex(_op(transa), _op(transb), pth, M, N, K, alpha, _ptr(A), lda, _ptr(B),
                          ldb, beta, _ptr(C), ldc, _stream(stream)))


def sgemm_ex_strided_batched(transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB,
                             beta, C, ldc, strideC, batch, path="simt", stream=None) -> None:
    pth = _PATHS.get(path, path) if isinstance(path, str) else int(path)
    _check(lib().sgemm_ex_strided_batched(_op(transa), _op(transb), pth, M, N, K, alpha, _ptr(A),
                                          lda, strideA, _ptr(B), ldb, strideB, beta, _ptr(C), ldc,
                                          strideC, batch, _stream(stream)))


def sgemm_fused(transa, transb, M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, bias=None,
                act="none", path="simt", stream=None) -> None:
    """C = act(alpha * op(A) op(B) + bias) + beta * C; act is 'none', 'relu', 'gelu',
    'gelu_tanh' or 'silu' (or its enum value); bias is an N-vector or None."""
    pth = _PATHS.get(path, path) if isinstance(path, str) else int(path)
    code = ACTIVATIONS[act] if isinstance(act, str) else int(act)
    _check(lib().sgemm_fused(_op(transa), _op(transb), pth, M, N, K, alpha, _ptr(A), lda,
                             _ptr(B), ldb, beta, _ptr(C), ldc, _ptr(bias), code, _stream(stream)))


def sgemm_fused_strided_batched(transa, transb, M, N, K, alpha, A, lda, strideA, B, ldb, strideB,
                                beta, C, ldc, strideC, batch, bias=None, act="none", path="simt",
                                stream=None) -> None:
    pth = _PATHS.get(path, path) if isinstance(path, str) else int(path)
    code = ACTIVATIONS[act] if isinstance(act, str) else int(act)
    _check(lib().sgemm_fused_strided_batched(_op(transa), _op(transb), pth, M, N, K, alpha,
                                             _ptr(A), lda, strideA, _ptr(B), ldb, strideB, beta,
                                             _ptr(C), ldc, strideC, batch, _ptr(bias), code,
                                             _stream(stream)))


def _host_ptr(x):
    if x is None or isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):  # a CPU torch tensor (pinned or not)
        if x.is_cuda:
            raise TypeError("sgemm_host takes host tensors")
        if str(x.dtype) != "torch.float32":
            raise TypeError("tensor arguments must be float32")
        return x.data_ptr()
    import numpy as np
    a = x if isinstance(x, np.ndarray) else np.asarray(x)
    if a.dtype != np.float32:
        raise TypeError("arrays must be float32")
    return a.ctypes.data


def sgemm_host(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """C = alpha * A.B + beta * C with host-memory operands (numpy arrays, CPU tensors or
    addresses); returns when C holds the result. Pinned memory lets copies overlap compute."""
    _check(lib().sgemm_host(M, N, K, alpha, _host_ptr(A), lda, _host_ptr(B), ldb, beta,
                            _host_ptr(C), ldc, _stream(stream)))


def sgemm_noalloc(M, N, K, alpha, A, lda, B, ldb, beta, C, ldc, stream=None) -> None:
    """sgemm() that allocates no device memory (its scratch is a static array in the library)."""
    _check(lib().sgemm_noalloc(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, beta, _ptr(C), ldc,
                               _stream(stream)))


def sgemm_status_string(status: int) -> str:
    return lib().sgemm_status_string(status).decode()


def sgemm_last_error() -> str:
    return (lib().sgemm_last_error() or b"").decode()


def sgemm_device_status(stream=None) -> int:
    """Synchronises ``stream``; returns the status code (does not raise)."""
    return lib().sgemm_device_status(_stream(stream))


def sgemm_release_workspace() -> None:
    _check(lib().sgemm_release_workspace())


def sgemm_num_configs() -> int:
    return lib().sgemm_num_configs()


def sgemm_config_name(i: int) -> str | None:
    name = lib().sgemm_config_name(i)
    return None if name is None else name.decode()


def sgemm_select_config(M, N, K, alpha, A, lda, B, ldb, C, ldc, batch=1) -> int:
    return lib().sgemm_select_config(M, N, K, alpha, _ptr(A), lda, _ptr(B), ldb, _ptr(C), ldc,
                                     batch)


def sgemm_force_config(i: int) -> None:
    _check(lib().sgemm_force_config(i))


def sgemm_selftest_bounded_wait(which: int, stream=None) -> None:
    """Queue a kernel whose bounded wait expires (failure-path test); see include/sgemm.h."""
    _check(lib().sgemm_selftest_bounded_wait(which, _stream(stream)))


def _side_stream(torch, device, queue):
    """The stream with the address `queue` (None: the current one) as a torch stream if it is not the
    current stream of `device`, else None."""
    if queue is None or queue == torch._C._cuda_getCurrentRawStream(device.index):
        return None
    if queue in (0, 1):  # the legacy default stream's two addresses
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(queue, device=device)


def _empty(torch, side, shape, dtype, device):
    """An output. On a side stream its memory comes from that stream's pool, so that no pending work
    of the current stream still uses it, and is kept while the current stream may use it."""
    if side is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(side):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _in_use(side, *tensors):
    """The tensors' memory is not handed out again before the side stream is done with it."""
    for t in tensors:
        if t is not None:
            t.record_stream(side)


def matmul(A, B, C=None, alpha: float = 1.0, beta: float = 0.0, tensor_cores: bool = False,
           stream=None):
    """torch convenience: row-major 2-D CUDA float32 tensors, returns C (allocated if None).

    Rows must be contiguous (stride(1) == 1); the row stride is the leading dimension. With a
    ``stream`` other than the current one, the inputs must be ready there and the caller orders
    later uses of C after it; no tensor's memory is handed out again before the call is done.
    """
    import torch
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError("matmul expects A (M x K) and B (K x N)")
    M, K = A.shape
    N = B.shape[1]
    side = None
    if stream is not None and A.is_cuda:
        side = _side_stream(torch, A.device, _stream(stream))
    if C is None:
        C = _empty(torch, side, (M, N), torch.float32, A.device)
        beta = 0.0
    for t in (A, B, C):
        if t.stride(1) != 1 and t.shape[1] > 1:
            raise ValueError("rows must be contiguous")
    if side is not None:
        _in_use(side, A, B, C)
    fn = sgemm_3xtf32 if tensor_cores else sgemm
    fn(M, N, K, alpha, A, max(A.stride(0), 1), B, max(B.stride(0), 1), beta, C,
       max(C.stride(0), 1), stream)
    return C


# ---- layer operators on 16-bit values ------------------------------------------------------------
#
# A call on a small layer costs the GPU a few microseconds, so these wrappers keep the host's share
# small: each tensor is looked at once, and the stream is read without building a Stream object.
#
# With a `stream` other than the current one, the inputs must be ready on it and the caller orders
# later uses of the outputs after it, as for any work on a side stream. The memory of a call's
# tensors is not handed out again before both streams are done with it, whenever they are dropped.

def _dtype_code(dtype) -> int:
    return dtype if isinstance(dtype, int) else _DTYPES.get(str(dtype), -1)


def _act_code(act) -> int:
    return ACTIVATIONS[act] if isinstance(act, str) else int(act)


def _ptr_as(x, names):
    """Address of a CUDA tensor whose dtype is one of `names` (or an address, or None)."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_cuda:
        raise TypeError("tensor arguments must live on a CUDA device")
    if str(x.dtype) not in names:
        raise TypeError(f"expected {' or '.join(names)}, got {x.dtype}")
    return x.data_ptr()


_NAMES16 = {SGEMM_DTYPE_BF16: ("torch.bfloat16",), SGEMM_DTYPE_F16: ("torch.float16",)}


def sgemm_linear(dtype, transw, M, N, K, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, Z=None, ldz=0,
                 stream=None) -> None:
    """Z = X op(W) + bias, Y = act(Z) + R on bfloat16 or half matrices (asynchronous on
    ``stream``); dtype is 'bf16' / 'f16', a torch dtype or the enum value. See
    include/sgemm.h."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_linear(dt, _op(transw), M, N, K, _ptr_as(X, names), ldx, _ptr_as(W, names),
                              ldw, _ptr_as(bias, names), _act_code(act), _ptr_as(R, names), ldr,
                              _ptr_as(Y, names), ldy, _ptr_as(Z, names), ldz, _stream(stream)))


def sgemm_linear_backward(dtype, transw, M, N, K, dY, lddy, Z, ldz, act, X, ldx, W, ldw, dX, lddx,
                          dW, lddw, db, stream=None) -> None:
    """The gradients of sgemm_linear (see include/sgemm.h); dX, dW and db may be None."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_linear_backward(dt, _op(transw), M, N, K, _ptr_as(dY, names), lddy,
                                       _ptr_as(Z, names), ldz, _act_code(act), _ptr_as(X, names),
                                       ldx, _ptr_as(W, names), ldw, _ptr_as(dX, names), lddx,
                                       _ptr_as(dW, names), lddw, _ptr(db), _stream(stream)))


def sgemm_moe(dtype, act, T, E, topk, D, F, X, ldx, Wr, ldwr, Wgate, Wup, ldu, strideu, Wdown, ldd,
              strided, renormalize, active, R, ldr, Y, ldy, topk_index=None, topk_weight=None,
              stream=None) -> None:
    """A whole mixture-of-experts layer for up to 64 tokens (see include/sgemm.h)."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_moe(dt, _act_code(act), T, E, topk, D, F, _ptr_as(X, names), ldx,
                           _ptr_as(Wr, names), ldwr, _ptr_as(Wgate, names), _ptr_as(Wup, names),
                           ldu, strideu, _ptr_as(Wdown, names), ldd, strided,
                           int(bool(renormalize)), _ptr_as(active, ("torch.bool", "torch.uint8")),
                           _ptr_as(R, names), ldr, _ptr_as(Y, names), ldy,
                           _ptr_as(topk_index, ("torch.int32",)),
                           _ptr_as(topk_weight, ("torch.float32",)), _stream(stream)))


_INT8, _FLOAT, _LABELS = ("torch.int8",), ("torch.float32",), ("torch.int64",)


def sgemm_checkpoint8(dtype, M, N, X, ldx, Q, ldq, S, lds, stream=None) -> None:
    """The 8-bit checkpoint (Q, S) of X (see include/sgemm.h)."""
    dt = _dtype_code(dtype)
    _check(lib().sgemm_checkpoint8(dt, M, N, _ptr_as(X, _NAMES16.get(dt, ())), ldx, _ptr_as(Q, _INT8), ldq,
                                   _ptr_as(S, _FLOAT), lds, _stream(stream)))


def sgemm_restore8(dtype, M, N, Q, ldq, S, lds, X, ldx, stream=None) -> None:
    """X restored from its 8-bit checkpoint (see include/sgemm.h)."""
    dt = _dtype_code(dtype)
    _check(lib().sgemm_restore8(dt, M, N, _ptr_as(Q, _INT8), ldq, _ptr_as(S, _FLOAT), lds,
                                _ptr_as(X, _NAMES16.get(dt, ())), ldx, _stream(stream)))


def sgemm_linear_checkpoint8(dtype, transw, M, N, K, X, ldx, W, ldw, bias, act, R, ldr, Y, ldy, Zq, ldzq,
                             Zs, ldzs, stream=None) -> None:
    """sgemm_linear with the pre-activation kept as an 8-bit checkpoint (see include/sgemm.h)."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_linear_checkpoint8(dt, _op(transw), M, N, K, _ptr_as(X, names), ldx,
                                          _ptr_as(W, names), ldw, _ptr_as(bias, names), _act_code(act),
                                          _ptr_as(R, names), ldr, _ptr_as(Y, names), ldy,
                                          _ptr_as(Zq, _INT8), ldzq, _ptr_as(Zs, _FLOAT), ldzs,
                                          _stream(stream)))


def sgemm_linear_backward_checkpoint8(dtype, transw, M, N, K, dY, lddy, Zq, ldzq, Zs, ldzs, act, Xq, ldxq,
                                      Xs, ldxs, W, ldw, dX, lddx, dW, lddw, db, stream=None) -> None:
    """The gradients of sgemm_linear from 8-bit checkpoints of X and Z (see include/sgemm.h)."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_linear_backward_checkpoint8(
        dt, _op(transw), M, N, K, _ptr_as(dY, names), lddy, _ptr_as(Zq, _INT8), ldzq, _ptr_as(Zs, _FLOAT),
        ldzs, _act_code(act), _ptr_as(Xq, _INT8), ldxq, _ptr_as(Xs, _FLOAT), ldxs, _ptr_as(W, names), ldw,
        _ptr_as(dX, names), lddx, _ptr_as(dW, names), lddw, _ptr(db), _stream(stream)))


def sgemm_cross_entropy(dtype, transw, T, V, D, X, ldx, W, ldw, labels, loss, lse, stream=None) -> None:
    """Softmax cross entropy of a vocabulary head (see include/sgemm.h); loss or lse may be None."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_cross_entropy(dt, _op(transw), T, V, D, _ptr_as(X, names), ldx, _ptr_as(W, names), ldw,
                                     _ptr_as(labels, _LABELS), _ptr_as(loss, _FLOAT), _ptr_as(lse, _FLOAT),
                                     _stream(stream)))


def sgemm_cross_entropy_backward(dtype, transw, T, V, D, dloss, incd, X, ldx, W, ldw, labels, lse, dX, lddx,
                                 dW, lddw, stream=None) -> None:
    """The gradients of sgemm_cross_entropy (see include/sgemm.h); dX or dW may be None."""
    dt = _dtype_code(dtype)
    names = _NAMES16.get(dt, ())
    _check(lib().sgemm_cross_entropy_backward(dt, _op(transw), T, V, D, _ptr_as(dloss, _FLOAT), incd,
                                              _ptr_as(X, names), ldx, _ptr_as(W, names), ldw,
                                              _ptr_as(labels, _LABELS), _ptr_as(lse, _FLOAT),
                                              _ptr_as(dX, names), lddx, _ptr_as(dW, names), lddw,
                                              _stream(stream)))


_torch = None
_CODES: dict = {}


def _setup():
    """torch, imported on first use (the C ABI's wrappers above work without it)."""
    global _torch
    import torch
    _CODES[torch.bfloat16] = SGEMM_DTYPE_BF16
    _CODES[torch.float16] = SGEMM_DTYPE_F16
    _torch = torch
    return torch


def _begin(x):
    """(torch, dtype, device, dtype code) of a call, from its first tensor."""
    torch = _torch or _setup()
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"expected a bfloat16 or float16 tensor, got {x.dtype}")
    return torch, x.dtype, x.device, code


def _queue(torch, device, stream):
    """(address, side stream or None) of a call's stream; the tensors must be on the calling thread's
    current device."""
    index = device.index
    if device.type != "cuda":
        raise TypeError("tensor arguments must live on a CUDA device")
    if index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index), None
    queue = stream if isinstance(stream, int) else stream.cuda_stream
    return queue, _side_stream(torch, device, queue)


def _matrix(t, rows, cols, dtype, device, what):
    """(address, leading dimension) of a rows x cols matrix of the call's type and device."""
    if t.shape != (rows, cols):
        raise ValueError(f"{what} must have shape {(rows, cols)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{what} is {t.dtype}: every matrix of a call has one 16-bit type")
    if t.device != device:
        raise ValueError("the tensors of a call must be on one device")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    return t.data_ptr(), (ld if rows > 1 else max(ld, cols, 1))


def _vector(t, n, device, what):
    if t.shape != (n,):
        raise ValueError(f"{what} must have shape {(n,)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError("the tensors of a call must be on one device")
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _weight_shape(weight, transw):
    """(N, K, transw code) of a weight stored N x K ('T') or K x N ('N')."""
    if weight.dim() != 2:
        raise ValueError("weight must be 2-D")
    a, b = weight.shape
    op = SGEMM_OP_T if transw == "T" else _op(transw)
    return (a, b, op) if op == SGEMM_OP_T else (b, a, op)


class Checkpoint8:
    """A matrix of 16-bit values kept in 8 bits: int8 ``codes``, a float32 ``scale`` for each 64 columns
    of a row, and the type that it is restored to (include/sgemm.h has the format). One that this
    library made has both in one buffer, of which ``codes`` and ``scale`` are views."""
    __slots__ = ("shape", "dtype", "device", "_codes", "_scale", "_buffer", "_ldq")

    def __init__(self, codes, scale, dtype):
        self.shape, self.dtype, self.device = tuple(codes.shape), dtype, codes.device
        self._codes, self._scale, self._buffer, self._ldq = codes, scale, None, 0

    @classmethod
    def _make(cls, torch, side, rows, cols, dtype, device):
        """A new one, codes in rows of whole 16 bytes; its scales follow them."""
        self = cls.__new__(cls)
        ldq = (cols + 15) // 16 * 16
        self.shape, self.dtype, self.device, self._codes, self._ldq = (rows, cols), dtype, device, None, ldq
        self._buffer = _empty(torch, side, (rows * (ldq + (cols + 63) // 64 * 4),), torch.int8, device)
        return self

    def _views(self):
        rows, cols = self.shape
        at = rows * self._ldq
        self._codes = self._buffer[:at].view(rows, self._ldq)[:, :cols]
        self._scale = self._buffer[at:].view(_torch.float32).view(rows, (cols + 63) // 64)

    @property
    def codes(self):
        if self._codes is None:
            self._views()
        return self._codes

    @property
    def scale(self):
        if self._codes is None:
            self._views()
        return self._scale

    def __repr__(self):
        return f"Checkpoint8(shape={self.shape}, dtype={self.dtype}, device={self.device})"

    def _tensors(self):
        return (self._codes, self._scale) if self._buffer is None else (self._buffer,)

    def _pointers(self, rows, cols, dtype, device, what):
        """(codes, ldq, scale, lds) of a rows x cols checkpoint of the call's type and device."""
        blocks = (cols + 63) // 64
        if self.shape != (rows, cols):
            raise ValueError(f"{what} must be a checkpoint of shape {(rows, cols)}, got {self.shape}")
        if self.dtype is not dtype:
            raise TypeError(f"{what} is a checkpoint of {self.dtype}: every matrix of a call has one 16-bit type")
        if self._buffer is not None:
            if self.device != device:
                raise ValueError("the tensors of a call must be on one device")
            at = self._buffer.data_ptr()
            return at, self._ldq or 1, at + rows * self._ldq, blocks or 1
        codes, scale = self._codes, self._scale
        if scale.shape != (rows, blocks):
            raise ValueError(f"{what}: scales must have shape {(rows, blocks)}, got {tuple(scale.shape)}")
        if codes.dtype is not _torch.int8 or scale.dtype is not _torch.float32:
            raise TypeError(f"{what}: a checkpoint has int8 codes and float32 scales")
        if codes.device != device or scale.device != device:
            raise ValueError("the tensors of a call must be on one device")
        (ldq, inner_q), (lds, inner_s) = codes.stride(), scale.stride()
        if (inner_q != 1 and cols > 1) or (inner_s != 1 and blocks > 1):
            raise ValueError(f"{what}: rows must be contiguous")
        if rows <= 1 or cols == 0:
            ldq, lds = max(ldq, cols, 1), max(lds, blocks, 1)
        return codes.data_ptr(), ldq, scale.data_ptr(), lds


def checkpoint8(x, stream=None):
    """torch convenience: the ``Checkpoint8`` of a 2-D bfloat16 or half CUDA tensor with contiguous
    rows: 1.06 bytes a value, each within a 254th of the largest of its 64."""
    torch, dtype, device, code = _begin(x)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, N = x.shape
    px, ldx = _matrix(x, M, N, dtype, device, "x")
    queue, side = _queue(torch, device, stream)
    c = Checkpoint8._make(torch, side, M, N, dtype, device)
    if side is not None:
        _in_use(side, x)
    status = (_lib or lib()).sgemm_checkpoint8(code, M, N, px, ldx, *c._pointers(M, N, dtype, device, "x"), queue)
    if status:
        _check(status)
    return c


def restore8(checkpoint, stream=None):
    """torch convenience: the matrix that a ``Checkpoint8`` stands for, in its 16-bit type."""
    torch, dtype, device, code = _begin(checkpoint)
    if len(checkpoint.shape) != 2:
        raise ValueError("a checkpoint's codes must be 2-D")
    M, N = checkpoint.shape
    saved = checkpoint._pointers(M, N, dtype, device, "the argument")
    queue, side = _queue(torch, device, stream)
    x = _empty(torch, side, (M, N), dtype, device)
    if side is not None:
        _in_use(side, *checkpoint._tensors())
    status = (_lib or lib()).sgemm_restore8(code, M, N, *saved, x.data_ptr(), max(N, 1), queue)
    if status:
        _check(status)
    return x


def linear(x, weight, bias=None, act="none", residual=None, transw="T", save_pre=False, out=None,
           stream=None):
    """torch convenience: act(x op(weight) + bias) + residual on 2-D bfloat16 or half CUDA
    tensors with contiguous rows. ``transw='T'`` takes a weight stored out x in (as
    torch.nn.Linear keeps it), 'N' one stored in x out. Returns y, or (y, pre) with the
    pre-activation that ``linear_backward`` reads when ``save_pre`` (as a ``Checkpoint8`` for
    ``save_pre='8bit'``). ``out`` may be ``residual`` itself. No gradient is recorded, whether or not the inputs require one
    (``Linear`` in examples/feed_forward.py does that)."""
    if isinstance(save_pre, str) and save_pre != "8bit":
        raise ValueError("save_pre is True, False or '8bit'")
    torch, dtype, device, code = _begin(x)
    N, K, op = _weight_shape(weight, transw)
    M = x.shape[0]
    px, ldx = _matrix(x, M, K, dtype, device, "x")
    pw, ldw = _matrix(weight, *weight.shape, dtype, device, "weight")
    pb = pr = pz = None
    ldr = 0
    if bias is not None:
        if bias.dtype is not dtype:
            raise TypeError(f"bias is {bias.dtype}: every matrix of a call has one 16-bit type")
        pb = _vector(bias, N, device, "bias")
    if residual is not None:
        pr, ldr = _matrix(residual, M, N, dtype, device, "residual")
    if out is not None:
        py, ldy = _matrix(out, M, N, dtype, device, "out")
    queue, side = _queue(torch, device, stream)
    if out is None:
        out, ldy = _empty(torch, side, (M, N), dtype, device), max(N, 1)
        py = out.data_ptr()
    if save_pre == "8bit":
        pre = Checkpoint8._make(torch, side, M, N, dtype, device)
    elif save_pre:
        pre = _empty(torch, side, (M, N), dtype, device)
        pz = pre.data_ptr()
    if side is not None:
        _in_use(side, x, weight, bias, residual, out)
    if save_pre == "8bit":
        status = (_lib or lib()).sgemm_linear_checkpoint8(code, op, M, N, K, px, ldx, pw, ldw, pb, _act_code(act),
                                                          pr, ldr, py, ldy,
                                                          *pre._pointers(M, N, dtype, device, "pre"), queue)
        if status:
            _check(status)
        return out, pre
    status = (_lib or lib()).sgemm_linear(code, op, M, N, K, px, ldx, pw, ldw, pb, _act_code(act), pr,
                                          ldr, py, ldy, pz, max(N, 1), queue)
    if status:
        _check(status)
    return (out, pre) if save_pre else out


def linear_backward(dy, x, weight, pre=None, act="none", transw="T", need_dx=True, need_dw=True,
                    need_db=True, stream=None):
    """torch convenience: (dx, dw, db) of ``linear`` from dy and the saved pre-activation
    (None for those not needed; db is float32). The residual's gradient is dy itself. x and pre
    may each be a ``Checkpoint8``: the results are those of the restored values."""
    saved = isinstance(x, Checkpoint8)
    if saved != isinstance(pre, Checkpoint8) and not (saved and pre is None):
        if saved:
            x, saved = restore8(x, stream=stream), False
        else:
            pre = restore8(pre, stream=stream)
    torch, dtype, device, code = _begin(x)
    N, K, op = _weight_shape(weight, transw)
    if saved:
        M = x.shape[0]
        px8 = x._pointers(M, K, dtype, device, "x")
        pz8 = ((None, max(N, 1), None, max(-(-N // 64), 1)) if pre is None
               else pre._pointers(M, N, dtype, device, "pre"))
    else:
        M = x.shape[0]
        px, ldx = _matrix(x, M, K, dtype, device, "x")
        pz, ldz = (None, 0) if pre is None else _matrix(pre, M, N, dtype, device, "pre")
    pw, ldw = _matrix(weight, *weight.shape, dtype, device, "weight")
    pg, ldg = _matrix(dy, M, N, dtype, device, "dy")
    queue, side = _queue(torch, device, stream)
    dx = dw = db = px_out = pw_out = pb_out = None
    if need_dx:
        dx = _empty(torch, side, (M, K), dtype, device)
        px_out = dx.data_ptr()
    if need_dw:
        dw = _empty(torch, side, weight.shape, dtype, device)
        pw_out = dw.data_ptr()
    if need_db:
        db = _empty(torch, side, (N,), torch.float32, device)
        pb_out = db.data_ptr()
    if side is not None:
        _in_use(side, dy, weight, *((*x._tensors(), *(pre._tensors() if pre else ())) if saved else (x, pre)))
    if saved:
        status = (_lib or lib()).sgemm_linear_backward_checkpoint8(
            code, op, M, N, K, pg, ldg, *pz8, _act_code(act), *px8, pw, ldw, px_out, max(K, 1), pw_out,
            max(weight.shape[1], 1), pb_out, queue)
        if status:
            _check(status)
        return dx, dw, db
    status = (_lib or lib()).sgemm_linear_backward(code, op, M, N, K, pg, ldg, pz, ldz, _act_code(act), px,
                                                   ldx, pw, ldw, px_out, max(K, 1), pw_out,
                                                   max(weight.shape[1], 1), pb_out, queue)
    if status:
        _check(status)
    return dx, dw, db


def _experts(w, E, rows, cols, dtype, device, what):
    """(address, leading dimension, expert stride) of an E x rows x cols tensor."""
    if w.shape != (E, rows, cols):
        raise ValueError(f"{what} must have shape {(E, rows, cols)}, got {tuple(w.shape)}")
    if w.dtype is not dtype:
        raise TypeError(f"{what} is {w.dtype}: every matrix of a call has one 16-bit type")
    if w.device != device:
        raise ValueError("the tensors of a call must be on one device")
    se, ld, inner = w.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{what}: rows must be contiguous")
    if rows <= 1:
        ld = max(ld, cols, 1)
    return w.data_ptr(), ld, (se if E > 1 else max(se, rows * ld))


def moe(x, router, w_gate, w_up, w_down, topk, act="silu", renormalize=True, active=None,
        residual=None, out=None, stream=None):
    """torch convenience: a whole mixture-of-experts layer for up to 64 tokens. x T x D, router
    E x D, w_gate (or None) and w_up E x F x D, w_down E x D x F, active T booleans or None.
    Returns (y, index, weight) with the chosen experts (int32) and their weights (float32),
    T x topk each. No gradient is recorded."""
    torch, dtype, device, code = _begin(x)
    if w_up.dim() != 3:
        raise ValueError("w_up must be 3-D (experts x hidden x width)")
    E, F, D = w_up.shape
    T = x.shape[0]
    px, ldx = _matrix(x, T, D, dtype, device, "x")
    pr, ldr = _matrix(router, E, D, dtype, device, "router")
    pu, ldu, su = _experts(w_up, E, F, D, dtype, device, "w_up")
    pg = pa = ps = None
    lds = 0
    if w_gate is not None:
        pg, *strides = _experts(w_gate, E, F, D, dtype, device, "w_gate")
        if strides != [ldu, su]:
            raise ValueError("w_gate and w_up must have the same strides")
    pd, ldd, sd = _experts(w_down, E, D, F, dtype, device, "w_down")
    if residual is not None:
        ps, lds = _matrix(residual, T, D, dtype, device, "residual")
    if active is not None:
        if active.dtype is not torch.bool and active.dtype is not torch.uint8:
            raise TypeError("active must be bool or uint8")
        pa = _vector(active, T, device, "active")
    if out is not None:
        py, ldy = _matrix(out, T, D, dtype, device, "out")
    queue, side = _queue(torch, device, stream)
    if out is None:
        out, ldy = _empty(torch, side, (T, D), dtype, device), max(D, 1)
        py = out.data_ptr()
    index = _empty(torch, side, (T, topk), torch.int32, device)
    weight = _empty(torch, side, (T, topk), torch.float32, device)
    if side is not None:
        _in_use(side, x, router, w_gate, w_up, w_down, active, residual, out)
    status = (_lib or lib()).sgemm_moe(code, _act_code(act), T, E, topk, D, F, px, ldx, pr, ldr, pg, pu, ldu,
                                       su, pd, ldd, sd, 1 if renormalize else 0, pa, ps, lds, py, ldy,
                                       index.data_ptr(), weight.data_ptr(), queue)
    if status:
        _check(status)
    return out, index, weight


def _labels(labels, T, device):
    if labels.dtype is not _torch.int64:
        raise TypeError(f"labels must be int64, got {labels.dtype}")
    return _vector(labels, T, device, "labels")


def cross_entropy(x, weight, labels, transw="T", stream=None):
    """torch convenience: (loss, lse), float32 per token, of the softmax over x op(weight) (x T x D;
    weight V x D for ``transw='T'``, D x V for 'N') at int64 labels. A label outside [0, V), such as
    -100, does not count: its loss is 0. The logits are not kept. No gradient is recorded
    (``cross_entropy_backward`` computes it from lse)."""
    torch, dtype, device, code = _begin(x)
    V, D, op = _weight_shape(weight, transw)
    T = x.shape[0]
    px, ldx = _matrix(x, T, D, dtype, device, "x")
    pw, ldw = _matrix(weight, *weight.shape, dtype, device, "weight")
    pl = _labels(labels, T, device)
    queue, side = _queue(torch, device, stream)
    loss = _empty(torch, side, (T,), torch.float32, device)
    lse = _empty(torch, side, (T,), torch.float32, device)
    if side is not None:
        _in_use(side, x, weight, labels)
    status = (_lib or lib()).sgemm_cross_entropy(code, op, T, V, D, px, ldx, pw, ldw, pl, loss.data_ptr(),
                                                 lse.data_ptr(), queue)
    if status:
        _check(status)
    return loss, lse


def cross_entropy_backward(dloss, x, weight, labels, lse, transw="T", need_dx=True, need_dw=True, stream=None):
    """torch convenience: (dx, dw) of ``cross_entropy`` from dloss (float32 per token, or one value
    expanded to that shape) and the lse that it returned; None for those not needed."""
    torch, dtype, device, code = _begin(x)
    V, D, op = _weight_shape(weight, transw)
    T = x.shape[0]
    px, ldx = _matrix(x, T, D, dtype, device, "x")
    pw, ldw = _matrix(weight, *weight.shape, dtype, device, "weight")
    pl = _labels(labels, T, device)
    for t, what in ((dloss, "dloss"), (lse, "lse")):
        if t.dtype is not torch.float32:
            raise TypeError(f"{what} must be float32, got {t.dtype}")
        if t.shape != (T,):
            raise ValueError(f"{what} must have shape {(T,)}, got {tuple(t.shape)}")
        if t.device != device:
            raise ValueError("the tensors of a call must be on one device")
    ps = _vector(lse, T, device, "lse")
    queue, side = _queue(torch, device, stream)
    dx = dw = pdx = pdw = None
    if need_dx:
        dx = _empty(torch, side, (T, D), dtype, device)
        pdx = dx.data_ptr()
    if need_dw:
        dw = _empty(torch, side, weight.shape, dtype, device)
        pdw = dw.data_ptr()
    if side is not None:
        _in_use(side, dloss, x, weight, labels, lse)
    status = (_lib or lib()).sgemm_cross_entropy_backward(code, op, T, V, D, dloss.data_ptr(), dloss.stride(0), px,
                                                          ldx, pw, ldw, pl, ps, pdx, D, pdw, weight.shape[1],
                                                          queue)
    if status:
        _check(status)
    return dx, dw
