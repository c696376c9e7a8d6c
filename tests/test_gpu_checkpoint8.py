"""GPU parity of the 8-bit checkpoints, of the linear layer that keeps one and of the gradients from
them, against the plain definitions in training_case.py and layer_case.py."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import layer_case as ref  # noqa: E402
import training_case as case  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def padded(t, pad, offset=0, fill=math.nan):
    """The same matrix as part of a wider buffer whose other values are `fill`."""
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset,), fill, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def same(a, b):
    return a.shape == b.shape and a.dtype == b.dtype and bool(((a == b) | ((a != a) & (b != b))).all())


def check_checkpoint(sg, x):
    c = sg.checkpoint8(x)
    codes, scale, restored = case.checkpoint_ref(x)
    assert same(c.codes, codes), (x.shape, int((c.codes != codes).sum()))
    assert same(c.scale, scale) and c.dtype is x.dtype
    assert same(sg.restore8(c), restored)
    assert sg.sgemm_device_status() == sg.SGEMM_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,N", [(1, 1), (1, 63), (3, 64), (2, 65), (7, 128), (5, 129), (33, 511), (64, 512), (130, 1000),
                                 (257, 1537), (1000, 72), (4099, 8), (9, 14336), (2, 70001)])
def test_sizes(sgemm_lib, dtype, M, N):
    check_checkpoint(sgemm_lib, normal(M + N, M, N, dtype=dtype))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (0, 1), (8, 8), (5, 3), (64, 1)])
@pytest.mark.parametrize("N", [200, 301, 512])
def test_strides_and_alignment(sgemm_lib, dtype, pad, offset, N):
    check_checkpoint(sgemm_lib, padded(normal(3, 37, N, dtype=dtype), pad, offset))


@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (7, 5), (8, 8), (16, 16), (24, 4), (64, 1)])
@pytest.mark.parametrize("N", [1, 40, 64, 191, 300])
def test_outputs_in_wider_buffers(sgemm_lib, pad, offset, N):
    """Codes, scales and the restored matrix at any address; what is around them stays."""
    sg, M = sgemm_lib, 21
    x = normal(5, M, N)
    codes, scale, restored = case.checkpoint_ref(x)
    blocks = scale.shape[1]
    q = padded(torch.zeros_like(codes), pad, offset, 99)
    s = padded(torch.zeros_like(scale), pad, offset)
    out = padded(torch.zeros_like(x), pad, offset)
    sg.sgemm_checkpoint8("bf16", M, N, x, N, q, N + pad, s, blocks + pad)
    sg.sgemm_restore8("bf16", M, N, q, N + pad, s, blocks + pad, out, N + pad)
    assert same(q, codes) and same(s, scale) and same(out, restored)
    for t, cols in ((q, N), (s, blocks), (out, N)):
        buf = t._base
        assert bool((buf[:offset] == 99).all() if t is q else torch.isnan(buf[:offset]).all())
        around = buf[offset:].view(M, cols + pad)[:, cols:]
        assert bool((around == 99).all() if t is q else torch.isnan(around).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_every_code_and_tie(sgemm_lib, dtype):
    """Blocks whose quotients are ties, or next to them, for many largest magnitudes."""
    g = torch.Generator(device="cuda").manual_seed(1)
    top = torch.randint(1, 2048 if dtype == torch.float16 else 256, (4000, 1), generator=g, device="cuda")
    v = (torch.rand(4000, 64, generator=g, device="cuda") * (2 * top + 1)).floor() - top
    v[:, 0] = top[:, 0]
    check_checkpoint(sgemm_lib, v.to(dtype))
    # ties: a = 127 / 2^k, values (q + 1/2) / 2^k
    for k in (0, 1, 5):
        q = torch.arange(-126, 127, device="cuda").float()
        v = torch.cat([(q + 0.5) / 2 ** k, torch.tensor([127.0 / 2 ** k], device="cuda")])
        rows = torch.stack([torch.cat([v[i::4], v[-1:]])[:64] for i in range(4)])
        rows[:, -1] = 127.0 / 2 ** k
        check_checkpoint(sgemm_lib, rows.to(dtype))


@pytest.mark.parametrize("dtype", DTYPES)
def test_range(sgemm_lib, dtype):
    """All bit patterns of the type, block by block of like and of unlike magnitudes."""
    bits = torch.arange(-32768, 32768, device="cuda", dtype=torch.int32).to(torch.int16)
    every = bits.view(dtype)
    check_checkpoint(sgemm_lib, every.view(-1, 64))
    g = torch.Generator(device="cuda").manual_seed(2)
    check_checkpoint(sgemm_lib, every[torch.randperm(65536, generator=g, device="cuda")].view(-1, 256))
    finite = every[torch.isfinite(every)]
    mixed = finite[torch.randperm(finite.numel(), generator=g, device="cuda")][:finite.numel() // 64 * 64]
    check_checkpoint(sgemm_lib, mixed.view(-1, 64))


@pytest.mark.parametrize("dtype", DTYPES)
def test_blocks_of_zeros_infinities_and_nan(sgemm_lib, dtype):
    x = normal(1, 6, 192, dtype=dtype)
    x[0] = 0.0
    x[1, 64:128] = 0.0
    x[2, 70] = math.inf
    x[3, 5] = -math.inf
    x[4, 191] = math.nan
    x[5, 64] = -0.0
    check_checkpoint(sgemm_lib, x)


def test_empty(sgemm_lib):
    sg = sgemm_lib
    for M, N in ((0, 5), (5, 0), (0, 0)):
        c = sg.checkpoint8(torch.zeros(M, N, dtype=torch.bfloat16, device="cuda"))
        assert c.codes.shape == (M, N) and c.scale.shape == (M, -(-N // 64))
        assert sg.restore8(c).shape == (M, N)


def test_offsets_past_32_bits(sgemm_lib):
    sg = sgemm_lib
    rows, pitch, N = 9, 1 << 29, 200
    x = normal(2, rows, N)
    codes, scale, restored = case.checkpoint_ref(x)
    q = torch.empty(rows * pitch, dtype=torch.int8, device="cuda").view(rows, pitch)[:, :N]
    s = torch.empty(rows, 4, device="cuda")
    sg.sgemm_checkpoint8("bf16", rows, N, x, N, q, pitch, s, 4)
    assert same(q, codes) and same(s, scale)
    del x
    out = torch.empty(rows * pitch, dtype=torch.bfloat16, device="cuda").view(rows, pitch)[:, :N]
    sg.sgemm_restore8("bf16", rows, N, q, pitch, s, 4, out, pitch)
    assert same(out, restored)
    c = sg.checkpoint8(out)  # and read from there
    again = case.checkpoint_ref(restored)
    assert same(c.codes, again[0])


def run_linear(sg, M, N, K, dtype, act, transw, bias, res, pad=0, offset=0, seed=0):
    """The values are linear's own, the checkpoint is that of the pre-activation that linear keeps."""
    x = padded(normal(seed, M, K, dtype=dtype), pad, offset)
    w = normal(seed + 1, *((N, K) if transw == "T" else (K, N)), dtype=dtype, scale=1 / math.sqrt(max(K, 1)))
    w = padded(w, pad, offset)
    b = normal(seed + 2, N, dtype=dtype) if bias else None
    r = padded(normal(seed + 3, M, N, dtype=dtype), pad, offset) if res else None
    y, pre = sg.linear(x, w, bias=b, act=act, residual=r, transw=transw, save_pre="8bit")
    y16, pre16 = sg.linear(x, w, bias=b, act=act, residual=r, transw=transw, save_pre=True)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert torch.equal(y, y16)
    codes, scale, restored = case.checkpoint_ref(pre16)
    assert same(pre.codes, codes) and same(pre.scale, scale)
    assert same(sg.restore8(pre), restored)
    ry, _, ytol, _ = ref.linear_ref(x, w, b, act, r, transw)
    assert ref.worst(y, ry, ytol) <= 1.0


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("M", [5, 384])
def test_linear_epilogues(sgemm_lib, dtype, act, M):
    run_linear(sgemm_lib, M, 640, 512, dtype, act, "T", True, True, seed=1)
    run_linear(sgemm_lib, M, 648, 512, dtype, act, "N", False, False, seed=2)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 129, 0), (64, 300, 72), (65, 2300, 136), (300, 1000, 264), (513, 577, 328),
                                   (1000, 3001, 200), (700, 520, 9001), (2048, 1536, 20000), (640, 2304, 256)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_linear_sizes(sgemm_lib, M, N, K, transw):
    run_linear(sgemm_lib, M, N, K, torch.bfloat16, "gelu", transw, True, True, seed=M)
    run_linear(sgemm_lib, M, N, K, torch.float16, "silu", transw, False, False, seed=N)


@pytest.mark.parametrize("M", [6, 300])
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (8, 1), (0, 5)])
def test_linear_strides(sgemm_lib, M, pad, offset):
    run_linear(sgemm_lib, M, 304, 264, torch.float16, "relu", "T", True, True, pad, offset, seed=3)


def test_linear_checkpoint_in_wider_buffers(sgemm_lib):
    sg = sgemm_lib
    for M in (9, 700):
        for N, pad, offset in ((640, 0, 0), (640, 16, 16), (633, 7, 3), (1000, 1, 0)):
            x, w = normal(1, M, 256), normal(2, N, 256, scale=1 / 16)
            _, want = sg.linear(x, w, act="silu", save_pre="8bit")
            blocks = -(-N // 64)
            q = padded(torch.zeros(M, N, dtype=torch.int8, device="cuda"), pad, offset, 99)
            s = padded(torch.zeros(M, blocks, device="cuda"), pad, offset)
            y = torch.empty(M, N, dtype=x.dtype, device="cuda")
            sg.sgemm_linear_checkpoint8("bf16", "T", M, N, 256, x, 256, w, 256, None, "silu", None, 0, y, N, q,
                                        N + pad, s, blocks + pad)
            assert same(q, want.codes) and same(s, want.scale)
            if pad:
                assert bool((q._base[offset:].view(M, N + pad)[:, N:] == 99).all())
                assert bool(torch.isnan(s._base[offset:].view(M, blocks + pad)[:, blocks:]).all())


def test_linear_nonfinite_blocks(sgemm_lib):
    sg = sgemm_lib
    for M in (8, 300):
        x, w = normal(1, M, 256), normal(2, 512, 256, scale=1 / 16)
        x[2, 3] = math.inf
        w[70] = math.nan
        _, pre = sg.linear(x, w, act="gelu", save_pre="8bit")
        _, pre16 = sg.linear(x, w, act="gelu", save_pre=True)
        codes, scale, _ = case.checkpoint_ref(pre16)
        assert same(pre.codes, codes) and same(pre.scale, scale)


def run_backward(sg, M, N, K, dtype, act, transw, pad=0, offset=0, seed=0):
    x8 = sg.checkpoint8(normal(seed, M, K, dtype=dtype))
    w = normal(seed + 1, *((N, K) if transw == "T" else (K, N)), dtype=dtype, scale=1 / math.sqrt(K))
    w = padded(w, pad, offset)
    dy = padded(normal(seed + 2, M, N, dtype=dtype), pad, offset)
    pre8 = None if act == "none" else sg.checkpoint8(normal(seed + 3, M, N, dtype=dtype))
    x, pre = sg.restore8(x8), None if pre8 is None else sg.restore8(pre8)
    got = sg.linear_backward(dy, x8, w, pre=pre8, act=act, transw=transw)
    want = sg.linear_backward(dy, x, w, pre=pre, act=act, transw=transw)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert all(torch.equal(a, b) for a, b in zip(got, want)), [int((a != b).sum()) for a, b in zip(got, want)]
    dx, dw, db, dxtol, dwtol, dbtol = ref.backward_ref(dy, x, w, pre, act, transw)
    for a, b, tol in zip(got, (dx, dw, db), (dxtol, dwtol, dbtol)):
        assert ref.worst(a, b, tol) <= 1.0
    return x8, w, dy, pre8, got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("transw", ["T", "N"])
def test_backward_activations(sgemm_lib, dtype, act, transw):
    run_backward(sgemm_lib, 300, 328, 264, dtype, act, transw, seed=4)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 200, 72), (33, 65, 129), (64, 1000, 520), (257, 301, 1537), (1000, 264, 333),
                                   (6338, 288, 80)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_backward_sizes(sgemm_lib, M, N, K, transw):
    run_backward(sgemm_lib, M, N, K, torch.bfloat16, "silu", transw, seed=M)


@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 1)])
def test_backward_strides(sgemm_lib, pad, offset):
    run_backward(sgemm_lib, 200, 304, 264, torch.float16, "gelu", "T", pad, offset)


def test_backward_parts_and_mixed_forms(sgemm_lib):
    sg = sgemm_lib
    for act in ("none", "gelu"):
        x8, w, dy, pre8, (dx, dw, db) = run_backward(sg, 130, 264, 200, torch.bfloat16, act, "T", seed=9)
        for need in ((1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0), (0, 0, 0)):
            got = sg.linear_backward(dy, x8, w, pre=pre8, act=act, need_dx=need[0], need_dw=need[1], need_db=need[2])
            for a, b, n in zip(got, (dx, dw, db), need):
                assert (a is None) if not n else torch.equal(a, b)
        if act != "none":  # one of the two in 16 bits
            for x, pre in ((sg.restore8(x8), pre8), (x8, sg.restore8(pre8))):
                assert all(torch.equal(a, b) for a, b in
                           zip(sg.linear_backward(dy, x, w, pre=pre, act=act), (dx, dw, db)))


def test_backward_degenerate(sgemm_lib):
    sg = sgemm_lib
    w = normal(1, 24, 16)
    none = torch.zeros(0, 16, dtype=w.dtype, device="cuda")
    dy = torch.zeros(0, 24, dtype=w.dtype, device="cuda")
    dx, dw, db = sg.linear_backward(dy, sg.checkpoint8(none), w, pre=sg.checkpoint8(dy), act="silu")
    assert dx.shape == (0, 16) and not dw.any() and not db.any()


def test_backward_against_differences(sgemm_lib):
    """The slope of the loss along random directions, with the forward pass in 64 bits on the restored
    values: what the gradients are the gradients of. Bound: dx, dw and db are each within 2^-8 of their norm
    (their rounding and dz's), and a central difference of step h is off by h^2 times a third derivative."""
    sg = sgemm_lib
    g = torch.Generator(device="cuda").manual_seed(0)
    M, N, K = 60, 90, 70
    x8, w = sg.checkpoint8(normal(1, M, K)), normal(2, N, K, scale=0.12)
    x = sg.restore8(x8).double()
    z = x @ w.double().t()
    pre8 = sg.checkpoint8(z.to(torch.bfloat16))
    dy = normal(3, M, N)
    dx, dw, _ = sg.linear_backward(dy, x8, w, pre=pre8, act="gelu_tanh")
    shift = sg.restore8(pre8).double() - z  # the slope is taken at the restored pre-activation

    def loss(x, w):
        return float((ref.act(x @ w.t() + shift, "gelu_tanh") * dy.double()).sum())

    for grad, at, other in ((dx, x, 0), (dw, w.double(), 1)):
        v = torch.randn(at.shape, generator=g, device="cuda", dtype=torch.float64)
        v /= v.norm()
        h = 1e-4
        args = [(at + h * v, w.double()), (at - h * v, w.double())] if other == 0 else [(x, at + h * v), (x, at - h * v)]
        slope = (loss(*args[0]) - loss(*args[1])) / (2 * h)
        assert abs(slope - float((grad.double() * v).sum())) <= 2.0 ** -7 * float(grad.double().norm())


def test_another_stream_and_graph(sgemm_lib):
    sg = sgemm_lib
    x, w, dy = normal(1, 300, 264), normal(2, 520, 264, scale=1 / 16), normal(3, 300, 520)

    def step(stream=None):
        x8 = sg.checkpoint8(x, stream=stream)
        y, pre = sg.linear(x, w, act="gelu", save_pre="8bit", stream=stream)
        return (y, sg.restore8(x8, stream=stream), *sg.linear_backward(dy, x8, w, pre=pre, act="gelu", stream=stream))

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = step()
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
        s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sg.sgemm_device_status() == sg.SGEMM_OK
