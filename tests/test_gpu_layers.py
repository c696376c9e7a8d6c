"""GPU parity of the layer operators (linear, its gradients, mixture of experts) against plain
64-bit definitions; tolerances are derived in layer_case.py."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import layer_case as ref  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def padded(t, pad, offset=0):
    """The same matrix as part of a wider buffer whose other values are NaN."""
    if pad == 0 and offset == 0:
        return t
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def run_linear(sg, M, N, K, dtype, act, transw, bias, res, pre, pad=0, offset=0, seed=0):
    x = padded(normal(seed, M, K, dtype=dtype), pad, offset)
    w = normal(seed + 1, *((N, K) if transw == "T" else (K, N)), dtype=dtype, scale=1 / math.sqrt(max(K, 1)))
    w = padded(w, pad, offset)
    b = normal(seed + 2, N, dtype=dtype) if bias else None
    r = padded(normal(seed + 3, M, N, dtype=dtype), pad, offset) if res else None
    out = padded(torch.zeros(M, N, dtype=dtype, device="cuda"), pad, offset)
    got = sg.linear(x, w, bias=b, act=act, residual=r, transw=transw, save_pre=pre, out=out)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    y, z = got if pre else (got, None)
    assert y is out
    if pad:  # nothing outside the matrix was written
        around = out._base.as_strided((M, pad), (N + pad, 1), offset + N)
        assert bool(torch.isnan(around).all())
    ry, rz, ytol, ztol = ref.linear_ref(x, w, b, act, r, transw)
    assert ref.worst(y, ry, ytol) <= 1.0, ("y", ref.worst(y, ry, ytol))
    if pre:
        assert ref.worst(z, rz, ztol) <= 1.0, ("z", ref.worst(z, rz, ztol))
    again = sg.linear(x, w, bias=b, act=act, residual=r, transw=transw)
    assert torch.equal(again, y), "two runs differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("M", [5, 384])
def test_linear_epilogues(sgemm_lib, dtype, act, transw, M):
    run_linear(sgemm_lib, M, 640, 512, dtype, act, transw, True, True, True, seed=1)
    run_linear(sgemm_lib, M, 640, 512, dtype, act, transw, False, False, False, seed=2)


ROWS = [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 48, 63, 64, 65, 96, 127, 128, 129, 160, 255, 256, 257, 300, 513]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("transw", ["T", "N"])
def test_linear_rows(sgemm_lib, M, transw):
    run_linear(sgemm_lib, M, 392, 328, torch.bfloat16, "silu", transw, True, True, True, seed=M)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (3, 1, 5), (1, 8, 8), (2, 129, 64), (130, 1, 70), (128, 256, 64),
                                   (16, 128, 16), (40, 24, 4099), (200, 136, 8), (77, 300, 2056),
                                   (256, 512, 64), (512, 256, 72), (257, 520, 136), (1, 4096, 64),
                                   (1000, 1000, 1000), (640, 2304, 256), (2048, 128, 4104)])
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_sizes(sgemm_lib, M, N, K, transw, dtype):
    run_linear(sgemm_lib, M, N, K, dtype, "gelu", transw, True, False, True, seed=5)


@pytest.mark.parametrize("M,N,K", [(1400, 1500, 5000), (700, 2999, 9001), (2048, 1536, 20000), (300, 260, 30000)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_linear_long_k_with_few_tiles(sgemm_lib, M, N, K, transw):
    run_linear(sgemm_lib, M, N, K, torch.bfloat16, "gelu", transw, True, True, True, seed=K)


@pytest.mark.parametrize("M", [1, 6, 33, 100, 300])
@pytest.mark.parametrize("N,K,pad,offset", [(301, 257, 0, 0), (304, 264, 3, 0), (304, 264, 8, 0), (304, 264, 8, 1),
                                            (304, 264, 0, 5), (303, 264, 1, 0), (304, 263, 1, 8)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_linear_strides_and_alignment(sgemm_lib, M, N, K, pad, offset, transw):
    run_linear(sgemm_lib, M, N, K, torch.float16, "relu", transw, True, True, True, pad, offset, seed=3)


def test_linear_residual_in_place(sgemm_lib):
    sg = sgemm_lib
    for M in (3, 200):
        x, w = normal(1, M, 256), normal(2, 320, 256, scale=1 / 16)
        r = normal(3, M, 320)
        want = sg.linear(x, w, act="silu", residual=r)
        sg.linear(x, w, act="silu", residual=r, out=r)
        assert torch.equal(r, want)


def test_linear_small_integers_are_exact(sgemm_lib):
    sg = sgemm_lib
    g = torch.Generator(device="cuda").manual_seed(0)
    for M in (1, 24, 130, 600):
        x = torch.randint(-2, 3, (M, 320), generator=g, device="cuda").half()
        w = torch.randint(-2, 3, (264, 320), generator=g, device="cuda").half()
        assert torch.equal(sg.linear(x, w).double(), x.double() @ w.double().t())


def test_linear_degenerate(sgemm_lib):
    sg = sgemm_lib
    b, r = normal(1, 24), normal(2, 5, 24)
    y = sg.linear(normal(3, 5, 0), normal(4, 24, 0), bias=b, act="gelu", residual=r)
    want, _, tol, _ = ref.linear_ref(torch.zeros(5, 1, device="cuda").bfloat16(),
                                     torch.zeros(24, 1, device="cuda").bfloat16(), b, "gelu", r, "T")
    assert ref.worst(y, want, tol) <= 1.0
    assert sg.linear(normal(1, 0, 8), normal(2, 24, 8)).shape == (0, 24)
    assert sg.linear(normal(1, 3, 8), normal(2, 0, 8)).shape == (3, 0)


@pytest.mark.parametrize("M", [4, 300])
def test_linear_nonfinite_rows_stay_apart(sgemm_lib, M):
    sg = sgemm_lib
    x, w, b = normal(1, M, 200), normal(2, 136, 200, scale=0.1), normal(3, 136)
    clean = sg.linear(x, w, bias=b, act="silu")
    x[1, 7] = math.nan
    x[2, 9] = math.inf
    y = sg.linear(x, w, bias=b, act="silu")
    keep = [i for i in range(M) if i not in (1, 2)]
    assert torch.equal(y[keep], clean[keep])
    assert bool(torch.isnan(y[1]).all())
    z = x.double() @ w.double().t() + b.double()
    assert bool((torch.isinf(y[2]) == (z[2] == math.inf)).all())


def test_linear_on_another_stream(sgemm_lib):
    sg = sgemm_lib
    x, w = normal(1, 64, 1024), normal(2, 512, 1024, scale=1 / 32)
    want = sg.linear(x, w, act="gelu")
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([sg.linear(x, w, act="gelu") for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for group in outs for o in group)


def test_linear_in_a_graph(sgemm_lib):
    sg = sgemm_lib
    x, w, b = normal(1, 4, 512), normal(2, 768, 512, scale=1 / 22), normal(3, 768)
    out = torch.empty(4, 768, dtype=x.dtype, device="cuda")
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        sg.linear(x, w, bias=b, act="silu", out=out)  # sizes the stream's workspace
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            sg.linear(x, w, bias=b, act="silu", out=out)
        for seed in (7, 8):
            x.copy_(normal(seed, 4, 512))
            graph.replay()
            torch.cuda.synchronize()
            want, _, tol, _ = ref.linear_ref(x, w, b, "silu", None, "T")
            assert ref.worst(out, want, tol) <= 1.0


# ---- gradients ---------------------------------------------------------------------------------

def run_backward(sg, M, N, K, dtype, act, transw, pad=0, offset=0, seed=0):
    x = padded(normal(seed, M, K, dtype=dtype), pad, offset)
    w = normal(seed + 1, *((N, K) if transw == "T" else (K, N)), dtype=dtype, scale=1 / math.sqrt(K))
    w = padded(w, pad, offset)
    pre = None if act == "none" else padded(normal(seed + 2, M, N, dtype=dtype, scale=1.5), pad, offset)
    dy = padded(normal(seed + 3, M, N, dtype=dtype, scale=0.1), pad, offset)
    dx, dw, db = sg.linear_backward(dy, x, w, pre=pre, act=act, transw=transw)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    rx, rw, rb, xt, wt, bt = ref.backward_ref(dy, x, w, pre, act, transw)
    for name, got, want, tol in (("dx", dx, rx, xt), ("dw", dw, rw, wt), ("db", db, rb, bt)):
        assert got.shape == want.shape
        assert ref.worst(got, want, tol) <= 1.0, (name, ref.worst(got, want, tol))
    again = sg.linear_backward(dy, x, w, pre=pre, act=act, transw=transw)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, dw, db))), "two runs differ"


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("transw", ["T", "N"])
def test_backward_activations(sgemm_lib, dtype, act, transw):
    run_backward(sgemm_lib, 200, 264, 392, dtype, act, transw, seed=1)


@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 64, 64), (2, 200, 72), (17, 129, 65), (64, 256, 1024), (100, 8, 2000),
                                   (129, 512, 8), (600, 312, 264), (2050, 136, 72), (1024, 1024, 512)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_backward_sizes(sgemm_lib, M, N, K, transw):
    run_backward(sgemm_lib, M, N, K, torch.bfloat16, "gelu", transw, seed=2)


@pytest.mark.parametrize("M,N,K", [(6000, 80, 288), (9000, 303, 72), (200, 9000, 260), (4000, 2000, 700)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_backward_long_k_with_few_tiles(sgemm_lib, M, N, K, transw):
    run_backward(sgemm_lib, M, N, K, torch.bfloat16, "silu", transw, seed=M)


@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1), (8, 3)])
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_backward_strides_and_alignment(sgemm_lib, pad, offset, transw, act):
    run_backward(sgemm_lib, 130, 264, 200, torch.float16, act, transw, pad, offset, seed=3)
    run_backward(sgemm_lib, 9, 264, 200, torch.float16, act, transw, pad, offset, seed=4)


def test_backward_parts_and_degenerate(sgemm_lib):
    sg = sgemm_lib
    dy, x, w, z = normal(1, 70, 96), normal(2, 70, 128), normal(3, 96, 128), normal(4, 70, 96)
    full = sg.linear_backward(dy, x, w, pre=z, act="silu")
    for i, need in enumerate(("need_dx", "need_dw", "need_db")):
        flags = {n: n == need for n in ("need_dx", "need_dw", "need_db")}
        part = sg.linear_backward(dy, x, w, pre=z, act="silu", **flags)
        assert torch.equal(part[i], full[i])
        assert all(p is None for j, p in enumerate(part) if j != i)
    dx, dw, db = sg.linear_backward(dy[:0], x[:0], w, pre=z[:0], act="silu")
    assert dx.shape == (0, 128) and not bool(dw.any()) and not bool(db.any())
    dx, dw, db = sg.linear_backward(normal(1, 70, 0), x, normal(3, 0, 128), pre=normal(4, 70, 0), act="silu")
    assert not bool(dx.any()) and dw.shape == (0, 128) and db.shape == (0,)


def test_backward_closed_relu_gate_stops_infinity(sgemm_lib):
    sg = sgemm_lib
    dy, x, w, z = normal(1, 40, 64), normal(2, 40, 72), normal(3, 64, 72), normal(4, 40, 64)
    z[3, 5] = -1.0
    want = sg.linear_backward(dy, x, w, pre=z, act="relu")
    dy[3, 5] = math.inf
    got = sg.linear_backward(dy, x, w, pre=z, act="relu")
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("act", ACTS)
def test_backward_against_differences(sgemm_lib, act):
    """dLoss along a direction, from central differences of the 64-bit forward pass with
    Loss = sum(c * Y): the truncation error is O(step^2) (1e-4 relative is generous at step 1e-3
    and unit curvature) and the gradients' own rounding is at most their tolerances."""
    sg = sgemm_lib
    M, N, K = 48, 40, 56
    dt = torch.float16
    x, w, b = normal(1, M, K, dtype=dt), normal(2, N, K, dtype=dt, scale=1 / 8), normal(3, N, dtype=dt)
    _, z = sg.linear(x, w, bias=b, act=act, save_pre=True)
    if act == "relu":  # away from the kink, where differences do not converge
        assert float((x.double() @ w.double().t() + b.double()).abs().min()) > 0
    c = normal(4, M, N, dtype=dt)
    grads = sg.linear_backward(c, x, w, pre=z, act=act)
    _, _, _, xt, wt, bt = ref.backward_ref(c, x, w, z, act, "T")
    # z itself was rounded: its slope moves by at most |act''| <= 2 times u |z|
    curve = 0.0 if act in ("none", "relu") else 2.0
    zerr = (curve * ref.U[dt] * z.double().abs()) * c.double().abs()
    extra = (zerr @ w.double().abs(), zerr.t() @ x.double().abs(), zerr.sum(0))
    base = [t.double() for t in (x, w, b)]
    for i, tol in enumerate((xt, wt, bt)):
        v = torch.sign(normal(10 + i, *base[i].shape)).double()
        step = 1e-6 if act == "relu" else 1e-3

        def loss(s):
            p = list(base)
            p[i] = p[i] + s * v
            return float((c.double() * ref.act(p[0] @ p[1].t() + p[2], act)).sum())

        want = (loss(step) - loss(-step)) / (2 * step)
        got = float((grads[i].double() * v).sum())
        bound = float((tol + extra[i]).sum()) + 1e-4 * float(grads[i].double().abs().sum())
        assert abs(got - want) <= bound


# ---- mixture of experts ---------------------------------------------------------------------------

def run_moe(sg, T, E, k, D, F, dtype, act="silu", gated=True, renormalize=True, active=None, residual=True,
            pad=0, offset=0, seed=0):
    x = padded(normal(seed, T, D, dtype=dtype), pad, offset)
    router = padded(normal(seed + 1, E, D, dtype=dtype, scale=1.5 / math.sqrt(D)), pad, offset)

    def experts(s, rows, cols):
        return padded(normal(s, E * rows, cols, dtype=dtype, scale=1 / math.sqrt(cols)), pad, offset) \
            .unflatten(0, (E, rows))

    gate = experts(seed + 2, F, D) if gated else None
    up, down = experts(seed + 3, F, D), experts(seed + 4, D, F)
    res = padded(normal(seed + 5, T, D, dtype=dtype), pad, offset) if residual else None
    out = padded(torch.zeros(T, D, dtype=dtype, device="cuda"), pad, offset)
    y, index, weight = sg.moe(x, router, gate, up, down, k, act=act, renormalize=renormalize,
                              active=active, residual=res, out=out)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    if pad:
        assert bool(torch.isnan(out._base.as_strided((T, pad), (D + pad, 1), offset + D)).all())
    ry, ri, rw, ytol, wtol = ref.moe_ref(x, router, gate, up, down, k, act, renormalize, active, res)
    assert torch.equal(index, ri)
    assert ref.worst(weight, rw, wtol + 1e-12) <= 1.0, ("weight", ref.worst(weight, rw, wtol + 1e-12))
    assert ref.worst(y, ry, ytol) <= 1.0, ("y", ref.worst(y, ry, ytol))
    again = sg.moe(x, router, gate, up, down, k, act=act, renormalize=renormalize, active=active,
                   residual=res)
    assert torch.equal(again[0], y) and torch.equal(again[1], index) and torch.equal(again[2], weight)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("renormalize", [True, False])
def test_moe_forms(sgemm_lib, dtype, act, gated, renormalize):
    run_moe(sgemm_lib, 6, 8, 2, 256, 384, dtype, act, gated, renormalize, seed=1)


@pytest.mark.parametrize("T", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64])
@pytest.mark.parametrize("E,k", [(8, 2), (60, 6)])
def test_moe_tokens(sgemm_lib, T, E, k):
    run_moe(sgemm_lib, T, E, k, 264, 200, torch.bfloat16, seed=T)


@pytest.mark.parametrize("T,E,k,D,F", [(1, 1, 1, 8, 8), (1, 1, 1, 1, 1), (4, 1, 1, 64, 64), (5, 4, 4, 128, 16),
                                       (64, 512, 16, 64, 32), (64, 16, 16, 128, 128), (2, 128, 8, 2048, 768),
                                       (3, 4, 1, 72, 4104), (1, 8, 2, 4096, 1024), (30, 3, 2, 1000, 136),
                                       (64, 2, 1, 512, 520)])
@pytest.mark.parametrize("gated", [True, False])
def test_moe_sizes(sgemm_lib, T, E, k, D, F, gated):
    run_moe(sgemm_lib, T, E, k, D, F, torch.float16, gated=gated, seed=2)


@pytest.mark.parametrize("T", [1, 7, 40])
@pytest.mark.parametrize("D,F,pad,offset", [(257, 301, 0, 0), (264, 304, 3, 0), (264, 304, 8, 0), (264, 304, 8, 1),
                                            (257, 304, 0, 0), (264, 301, 0, 0)])
def test_moe_strides_and_alignment(sgemm_lib, T, D, F, pad, offset):
    run_moe(sgemm_lib, T, 6, 2, D, F, torch.bfloat16, pad=pad, offset=offset, seed=3)


def test_moe_idle_slots(sgemm_lib):
    sg = sgemm_lib
    for T, seed in ((5, 1), (64, 2)):
        active = torch.arange(T, device="cuda") % 3 != 1
        run_moe(sg, T, 8, 2, 256, 192, torch.bfloat16, active=active, seed=seed)
    none = torch.zeros(4, dtype=torch.bool, device="cuda")
    run_moe(sg, 4, 8, 2, 256, 192, torch.bfloat16, active=none, seed=3)
    run_moe(sg, 4, 8, 2, 256, 192, torch.bfloat16, active=none, residual=False, seed=3)


def test_moe_nonfinite_rows_stay_apart(sgemm_lib):
    sg = sgemm_lib
    T, E, D, F = 9, 4, 200, 136
    x, router = normal(1, T, D), normal(2, E, D, scale=0.1)
    gate, up, down = normal(3, E, F, D, scale=0.1), normal(4, E, F, D, scale=0.1), normal(5, E, D, F, scale=0.1)
    clean = sg.moe(x, router, gate, up, down, 2)
    x[2] = math.nan
    x[5, 3] = math.inf
    y, index, weight = sg.moe(x, router, gate, up, down, 2)
    keep = [0, 1, 3, 4, 6, 7, 8]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(index[keep], clean[1][keep])
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(weight[2]).all())
    assert bool(((index >= 0) & (index < E)).all())
    # an idle slot's values are not used
    active = torch.ones(T, dtype=torch.uint8, device="cuda")
    active[2] = active[5] = 0
    y, index, weight = sg.moe(x, router, gate, up, down, 2, active=active)
    assert torch.equal(y[keep], clean[0][keep])
    assert not bool(y[2].any()) and not bool(weight[5].any()) and bool((index[2] == -1).all())


def test_moe_equal_scores_go_to_the_lowest_index(sgemm_lib):
    sg = sgemm_lib
    T, E, D, F = 3, 70, 64, 64
    x = normal(1, T, D)
    router = torch.zeros(E, D, dtype=x.dtype, device="cuda")
    up, down = normal(4, E, F, D, scale=0.1), normal(5, E, D, F, scale=0.1)
    _, index, weight = sg.moe(x, router, None, up, down, 5, act="relu", renormalize=False)
    assert index.tolist() == [[0, 1, 2, 3, 4]] * T
    assert torch.allclose(weight.double(), torch.full((T, 5), 1 / E, device="cuda", dtype=torch.float64), rtol=1e-6)
    _, index, _ = sg.moe(x, router, None, up, down, 16, act="relu")
    assert index.tolist() == [list(range(16))] * T


def test_moe_weights_of_other_experts_are_not_read_into_the_result(sgemm_lib):
    sg = sgemm_lib
    T, E, D, F = 2, 8, 128, 192
    x, router = normal(1, T, D), normal(2, E, D, scale=0.2)
    gate, up, down = normal(3, E, F, D, scale=0.1), normal(4, E, F, D, scale=0.1), normal(5, E, D, F, scale=0.1)
    y, index, _ = sg.moe(x, router, gate, up, down, 2)
    unused = [e for e in range(E) if e not in set(index.flatten().tolist())]
    for t in (gate, up, down):
        t[unused] = math.nan
    assert torch.equal(sg.moe(x, router, gate, up, down, 2)[0], y)


def test_moe_in_place_residual_streams_and_graph(sgemm_lib):
    sg = sgemm_lib
    T, E, D, F = 4, 8, 256, 320
    x, router = normal(1, T, D), normal(2, E, D, scale=0.1)
    gate, up, down = normal(3, E, F, D, scale=0.06), normal(4, E, F, D, scale=0.06), normal(5, E, D, F, scale=0.06)
    want = sg.moe(x, router, gate, up, down, 2, residual=x)[0]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append([sg.moe(x, router, gate, up, down, 2, residual=x)[0] for _ in range(4)])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for group in outs for o in group)
    with torch.cuda.stream(streams[0]):
        y = x.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=streams[0]):
            sg.moe(x, router, gate, up, down, 2, residual=y, out=y)
        y.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


# ---- offsets past 32 bits ------------------------------------------------------------------------------

@pytest.mark.parametrize("rows,pitch", [(12, 1 << 28), (300, 1 << 23)])
def test_linear_offsets_past_32_bits(sgemm_lib, rows, pitch):
    """x, residual, pre-activation and output as columns of one buffer whose last rows lie more than
    2^31 values in."""
    sg = sgemm_lib
    K, N = 264, 328
    assert rows * pitch > 1 << 31
    buf = torch.empty(rows, pitch, dtype=torch.bfloat16, device="cuda")
    x, r, out, dy, z = (buf[:, at:at + n] for at, n in ((0, K), (512, N), (1024, N), (1536, N), (2048, N)))
    x.copy_(normal(1, rows, K))
    r.copy_(normal(2, rows, N))
    w = normal(3, N, K, scale=1 / 16)
    sg.linear(x, w, act="silu", residual=r, out=out)
    want, _, tol, _ = ref.linear_ref(x, w, None, "silu", r, "T")
    assert ref.worst(out, want, tol) <= 1.0
    dy.copy_(normal(4, rows, N))
    z.copy_(normal(5, rows, N))
    got = sg.linear_backward(dy, x, w, pre=z, act="gelu")
    rx, rw, rb, xt, wt, bt = ref.backward_ref(dy, x, w, z, "gelu", "T")
    assert max(ref.worst(got[0], rx, xt), ref.worst(got[1], rw, wt), ref.worst(got[2], rb, bt)) <= 1.0
    assert sg.sgemm_device_status() == sg.SGEMM_OK


@pytest.mark.parametrize("shift", [0, 1])
def test_moe_expert_offsets_past_32_bits(sgemm_lib, shift):
    sg = sgemm_lib
    T, E, D, F, stride = 5, 4, 136, 72, (1 << 30) - 8 * 5
    buf = torch.empty(E * stride, dtype=torch.bfloat16, device="cuda")
    assert (E - 1) * stride > 1 << 31
    up = buf[shift:].as_strided((E, F, D), (stride, D, 1))
    gate = buf[1 << 20:].as_strided((E, F, D), (stride, D, 1), (1 << 20) + shift)
    down = buf.as_strided((E, D, F), (stride, F, 1), (1 << 21) + shift)
    for i, t in enumerate((up, gate, down)):
        t.copy_(normal(10 + i, *t.shape, scale=0.1))
    x, router = normal(1, T, D), normal(2, E, D, scale=0.2)
    y, index, weight = sg.moe(x, router, gate, up, down, 2)
    want, ri, rw, tol, wtol = ref.moe_ref(x, router, gate, up, down, 2, "silu", True, None, None)
    assert torch.equal(index, ri) and ref.worst(y, want, tol) <= 1.0
    assert sg.sgemm_device_status() == sg.SGEMM_OK
