"""GPU parity of the head's cross entropy and its gradient against the plain definitions in 64 bits;
tolerances are derived in training_case.py."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import training_case as case  # noqa: E402
from layer_case import worst  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def padded(t, pad, offset=0):
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def inputs(T, V, D, dtype=torch.bfloat16, transw="T", ignored=0.2, pad=0, offset=0, seed=0, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = padded(normal(seed + 1, T, D, dtype=dtype), pad, offset)
    w = normal(seed + 2, *((V, D) if transw == "T" else (D, V)), dtype=dtype, scale=spread / math.sqrt(D))
    w = padded(w, pad, offset)
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    labels[torch.rand(T, generator=g, device="cuda") < ignored] = -100
    dloss = torch.randn(T, generator=g, device="cuda") / max(T, 1)
    return x, w, labels, dloss


def check(sg, x, w, labels, dloss, transw="T"):
    loss, lse = sg.cross_entropy(x, w, labels, transw=transw)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    rloss, rlse, _, tol, ltol, _ = case.head_ref(x, w, labels, transw)
    assert worst(lse, rlse, ltol) <= 1.0, worst(lse, rlse, ltol)
    assert worst(loss, rloss, tol) <= 1.0, worst(loss, rloss, tol)
    given = rlse.float()
    dx, dw = sg.cross_entropy_backward(dloss, x, w, labels, given, transw=transw)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    rdx, rdw, dxtol, dwtol = case.head_grad_ref(dloss, x, w, labels, given, transw)
    assert worst(dx, rdx, dxtol) <= 1.0, worst(dx, rdx, dxtol)
    assert worst(dw, rdw, dwtol) <= 1.0, worst(dw, rdw, dwtol)
    V = w.shape[0] if transw == "T" else w.shape[1]
    skipped = (labels < 0) | (labels >= V)
    assert not bool(dx[skipped].any()) and not bool(loss[skipped].any())
    again = (*sg.cross_entropy(x, w, labels, transw=transw),
             *sg.cross_entropy_backward(dloss, x, w, labels, given, transw=transw))
    assert all(torch.equal(a, b) for a, b in zip((loss, lse, dx, dw), again)), "two runs differ"
    return loss, lse, dx, dw


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("T,V,D", [(1, 1, 1), (1, 2, 8), (2, 63, 16), (3, 64, 64), (5, 65, 72), (16, 257, 64), (31, 1000, 136),
                                   (32, 512, 64), (33, 4097, 200), (64, 1000, 512), (65, 300, 333), (127, 999, 64),
                                   (128, 2048, 256), (129, 515, 1537), (256, 256, 256), (257, 3001, 72), (300, 1003, 265),
                                   (513, 777, 128)])
def test_sizes(sgemm_lib, dtype, transw, T, V, D):
    x, w, labels, dloss = inputs(T, V, D, dtype, transw, seed=T + V)
    check(sgemm_lib, x, w, labels, dloss, transw)


@pytest.mark.parametrize("T,V,D", [(1, 32000, 512), (7, 50257, 128), (700, 30001, 200), (2, 131072, 64), (1500, 5000, 4104)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_large_vocabularies(sgemm_lib, T, V, D, transw):
    x, w, labels, dloss = inputs(T, V, D, torch.bfloat16, transw, seed=V)
    check(sgemm_lib, x, w, labels, dloss, transw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transw", ["T", "N"])
def test_pieces_of_tokens_and_vocabulary(sgemm_lib, dtype, transw):
    """More tokens than the forward pass takes at once, more logits than the gradient keeps at once."""
    x, w, labels, dloss = inputs(40000, 9001, 72, dtype, transw, seed=1)
    check(sgemm_lib, x, w, labels, dloss, transw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (8, 1), (0, 5), (1, 8)])
def test_strides_and_alignment(sgemm_lib, dtype, transw, pad, offset):
    for T, V, D in ((6, 301, 72), (300, 504, 200)):
        x, w, labels, dloss = inputs(T, V, D, dtype, transw, pad=pad, offset=offset, seed=3)
        check(sgemm_lib, x, w, labels, dloss, transw)


@pytest.mark.parametrize("pad,offset", [(0, 0), (3, 0), (8, 8), (8, 1)])
@pytest.mark.parametrize("transw", ["T", "N"])
def test_outputs_in_wider_buffers(sgemm_lib, pad, offset, transw):
    sg, (T, V, D) = sgemm_lib, (150, 500, 136)
    x, w, labels, dloss = inputs(T, V, D, transw=transw, seed=4)
    loss, lse, dx, dw = check(sg, x, w, labels, dloss, transw)
    lse = case.head_ref(x, w, labels, transw)[1].float()
    ox, ow = padded(torch.zeros_like(dx), pad, offset), padded(torch.zeros_like(dw), pad, offset)
    sg.sgemm_cross_entropy_backward("bf16", transw, T, V, D, dloss, 1, x, D, w, w.stride(0), labels, lse, ox, D + pad, ow,
                                    dw.shape[1] + pad)
    assert torch.equal(ox, dx) and torch.equal(ow, dw)
    for t in (ox, ow):
        assert bool(torch.isnan(t._base[:offset]).all())
        assert bool(torch.isnan(t._base[offset:].view(t.shape[0], -1)[:, t.shape[1]:]).all())


@pytest.mark.parametrize("T", [3, 200])
def test_labels(sgemm_lib, T):
    """Labels outside the vocabulary, and far outside; none that counts."""
    x, w, labels, dloss = inputs(T, 300, 64, ignored=0.0, seed=5)
    for bad in (-1, -100, 300, 1 << 31, 1 << 32, -(1 << 32), (1 << 63) - 1, -(1 << 63)):
        some = labels.clone()
        some[::2] = bad
        check(sgemm_lib, x, w, some, dloss)
    loss, lse, dx, dw = check(sgemm_lib, x, w, torch.full_like(labels, -100), dloss)
    assert not loss.any() and not dx.any() and not dw.any() and bool(torch.isfinite(lse).all())
    for v in (0, 63, 64, 255, 256, 299):  # one label for all
        check(sgemm_lib, x, w, torch.full_like(labels, v), dloss)


@pytest.mark.parametrize("dtype", DTYPES)
def test_certain_and_wide_logits(sgemm_lib, dtype):
    """Logits of hundreds, where all but one probability vanish."""
    for spread in (0.0, 20.0, 100.0):
        x, w, labels, dloss = inputs(140, 700, 128, dtype, seed=6, spread=spread)
        check(sgemm_lib, x, w, labels, dloss)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("scale", [1e-6, 1.0, 3e4])
def test_sizes_of_dloss(sgemm_lib, dtype, scale):
    """Each token's own, one value for all (expanded), zeros, and values far below the largest."""
    x, w, labels, _ = inputs(200, 700, 128, dtype, seed=7)
    w = (w.float() * 0.2).to(dtype)
    g = torch.Generator(device="cuda").manual_seed(1)
    if dtype == torch.float16 and scale < 1:
        scale = 1e-2  # (the outputs' own subnormals)
    if dtype == torch.float16 and scale > 1:
        scale = 1e3  # (dw is up to |dloss| times a few of x, and half ends at 65504)
    check(sgemm_lib, x, w, labels, torch.full((), scale, device="cuda").expand(200))
    check(sgemm_lib, x, w, labels, torch.zeros(200, device="cuda"))
    check(sgemm_lib, x, w, labels, scale * torch.rand(200, generator=g, device="cuda") ** 8)
    strided = torch.zeros(200, 3, device="cuda")
    strided[:, 1] = scale * torch.randn(200, generator=g, device="cuda").clamp(-1, 1)
    check(sgemm_lib, x, w, labels, strided[:, 1])


def test_half_keeps_small_probabilities(sgemm_lib):
    """A mean over many tokens of a flat distribution: |dz| of 1e-9 and less, far below half's smallest value,
    decides dw's norm together with the labels' entries, which are left out here."""
    sg = sgemm_lib
    T, V, D = 64, 20000, 64
    x, w, labels, _ = inputs(T, V, D, torch.float16, ignored=0.0, seed=8, spread=0.5)
    x = x.abs()
    labels = labels % 100
    dloss = torch.full((T,), 1e-2, device="cuda")
    _, lse = sg.cross_entropy(x, w, labels)
    _, dw = sg.cross_entropy_backward(dloss, x, w, labels, lse)
    _, want, _, tol = case.head_grad_ref(dloss, x, w, labels, lse, "T")
    assert worst(dw, want, tol) <= 1.0
    rest = want[100:]
    assert float((dw[100:].double() - rest).norm() / rest.norm()) < 0.02


def summing_error(x, w, labels, run):
    """What the label's logit may lose: the tensor cores cut their sum (to fp32, by less than a step) once per 16
    products, from zero in each run of `run` products; the runs are added with rounding, half a step each."""
    def step(v):
        return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-30))) - 23)

    products = x.double() * w.double()[labels]
    T, D = products.shape
    lost = torch.zeros(T, dtype=torch.float64, device=x.device)
    total = torch.zeros_like(lost)
    for r in range(0, D, run):
        part = torch.zeros_like(lost)
        for k in range(r, min(r + run, D), 16):
            grown = part + products[:, k:min(k + 16, r + run, D)].sum(1)
            lost += step(torch.maximum(part.abs(), grown.abs()))
            part = grown
        if r > 0:
            lost += step(total + part) / 2
        total = total + part
    return lost


@pytest.mark.parametrize("T", [1, 7, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_labels_that_are_all_but_certain(sgemm_lib, dtype, T):
    """1 - p at the labels is about 10^-4 and the gradient no larger, so that the logit's own error shows in it.
    A row of dX is off by (dloss 1): the label's logit's error (times p < 1) and expm1f's two steps of 1 - p, through
    the label's row of W; 2^-18 of each other p (a logit's error below 2^-19 and the exponential's); a rounding of each
    dz to 16 bits; and dX's own sum and rounding. z - lse is exact: the two are within a factor 2 of each other."""
    sg, (V, D) = sgemm_lib, (56, 704)
    u, tiny = case.U[dtype] * 1.001, case.TINY[dtype]
    g = torch.Generator(device="cuda").manual_seed(T)
    w = normal(1, V, D, dtype=dtype, scale=1.28 / math.sqrt(D))
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    x = (normal(2, T, D, dtype=dtype).float() + 8.5 * w[labels].float()).to(dtype)
    ones = torch.full((), 1.0, device="cuda").expand(T)
    z = x.double() @ w.double().t()
    exact = torch.logsumexp(z, 1).float()
    own = sg.cross_entropy(x, w, labels)[1]
    length = w.double().norm(dim=1)
    lost = summing_error(x, w, labels, 64)
    for lse in (exact, own):
        dx, _ = sg.cross_entropy_backward(ones, x, w, labels, lse)
        assert sg.sgemm_device_status() == sg.SGEMM_OK
        gap = z - lse.double()[:, None]
        dz = torch.exp(gap)
        dz.scatter_(1, labels[:, None], torch.expm1(gap.gather(1, labels[:, None])))
        ref = dz @ w.double()
        at = dz.gather(1, labels[:, None])[:, 0].abs()
        off = (2.0 ** -18 + u) * (dz.abs() @ length) + (lost + 2.0 ** -22 * at) * length[labels]
        off += case.ACC * (dz.abs() @ w.double().abs()).norm(dim=1) + u * ref.norm(dim=1) + tiny * math.sqrt(D) * (1 + V)
        ratio = (dx.double() - ref).norm(dim=1) / off
        assert bool((ratio <= 1.0).all()), ratio


def test_parts(sgemm_lib):
    sg = sgemm_lib
    for dtype, T in ((torch.bfloat16, 5), (torch.float16, 300)):
        x, w, labels, dloss = inputs(T, 500, 136, dtype, seed=9)
        loss, lse = sg.cross_entropy(x, w, labels)
        dx, dw = sg.cross_entropy_backward(dloss, x, w, labels, lse)
        a, none = sg.cross_entropy_backward(dloss, x, w, labels, lse, need_dw=False)
        assert torch.equal(a, dx) and none is None
        none, b = sg.cross_entropy_backward(dloss, x, w, labels, lse, need_dx=False)
        assert torch.equal(b, dw) and none is None
        only = torch.empty_like(lse)
        name = "bf16" if dtype == torch.bfloat16 else "f16"
        sg.sgemm_cross_entropy(name, "T", T, 500, 136, x, 136, w, 136, labels, None, only)
        assert torch.equal(only, lse)
        sg.sgemm_cross_entropy(name, "T", T, 500, 136, x, 136, w, 136, labels, only, None)
        assert torch.equal(only, loss)


def test_no_tokens(sgemm_lib):
    sg = sgemm_lib
    x, w = torch.zeros(0, 16, dtype=torch.bfloat16, device="cuda"), normal(1, 24, 16)
    labels, empty = torch.zeros(0, dtype=torch.int64, device="cuda"), torch.zeros(0, device="cuda")
    loss, lse = sg.cross_entropy(x, w, labels)
    assert loss.shape == (0,) and lse.shape == (0,)
    dx, dw = sg.cross_entropy_backward(empty, x, w, labels, empty)
    assert dx.shape == (0, 16) and dw.shape == (24, 16) and not dw.any()


def test_infinite_and_nan_logits(sgemm_lib):
    """A logit of -inf has no probability; +inf or NaN makes its own token's loss NaN and no other's. (Rows of
    the product cannot mix, so the rest is held to the definition.)"""
    sg = sgemm_lib
    T, V, D = 140, 700, 64
    x, w, labels, dloss = inputs(T, V, D, ignored=0.0, seed=10)
    x[:, 0] = 1.0
    x[5, 0] = -1.0
    w[:, 0] = 0.0
    w[64:130, 0] = -math.inf  # a whole part of 64 columns among them
    labels = torch.where((labels >= 64) & (labels < 130), 0, labels)
    loss, lse = sg.cross_entropy(x, w, labels)
    z = x.double() @ w.double().t()
    assert bool(torch.isnan(lse[5])) and bool(torch.isnan(loss[5]))
    keep = torch.arange(T, device="cuda") != 5
    want = torch.logsumexp(z[keep], 1)
    assert float((lse[keep].double() - want).abs().max()) < 1e-4
    x2, w2, labels2, _ = inputs(T, V, D, ignored=0.0, seed=11)
    x2[7, 3] = math.nan
    labels2[9] = -100
    x2[9, 3] = math.inf
    loss, lse = sg.cross_entropy(x2, w2, labels2)
    assert torch.nonzero(torch.isnan(loss))[:, 0].tolist() == [7]
    assert float(loss[9]) == 0.0
    dx, _ = sg.cross_entropy_backward(dloss, x2, w2, labels2, lse)
    assert torch.nonzero(torch.isnan(dx.float()).any(1))[:, 0].tolist() == [7]
    assert not dx[9].any()


@pytest.mark.parametrize("T", [3, 200])
def test_a_row_without_a_finite_logit(sgemm_lib, T):
    """All logits -inf: lse is -inf, the loss NaN, and the other rows are as without it."""
    sg = sgemm_lib
    x, w, labels, _ = inputs(T, 300, 64, ignored=0.0, seed=16)
    x[:, 0], w[:, 0] = 0.0, 1.0
    want, want_lse = sg.cross_entropy(x, w, labels)
    x[1, 0] = -math.inf
    loss, lse = sg.cross_entropy(x, w, labels)
    keep = torch.arange(T, device="cuda") != 1
    assert float(lse[1]) == -math.inf and bool(torch.isnan(loss[1]))
    assert torch.equal(loss[keep], want[keep]) and torch.equal(lse[keep], want_lse[keep])


def test_gradient_against_differences(sgemm_lib):
    """The slope of the weighted loss along random directions, the loss in 64 bits: |error| <= 2^-7 |gradient|
    (dz's rounding and the outputs'), a central difference's own being h^2."""
    sg = sgemm_lib
    x, w, labels, dloss = inputs(90, 400, 72, seed=12)
    _, lse = sg.cross_entropy(x, w, labels)
    dx, dw = sg.cross_entropy_backward(dloss, x, w, labels, lse)
    g = torch.Generator(device="cuda").manual_seed(0)

    def loss(x, w):
        z = x @ w.t()
        each = torch.logsumexp(z, 1) - z.gather(1, labels.clamp(min=0)[:, None])[:, 0]
        return float((each * dloss.double() * (labels >= 0)).sum())

    for grad, which in ((dx, 0), (dw, 1)):
        at = [x.double(), w.double()]
        v = torch.randn(at[which].shape, generator=g, device="cuda", dtype=torch.float64)
        v /= v.norm()
        up, down = list(at), list(at)
        up[which], down[which] = at[which] + 1e-4 * v, at[which] - 1e-4 * v
        slope = (loss(*up) - loss(*down)) / 2e-4
        assert abs(slope - float((grad.double() * v).sum())) <= 2.0 ** -7 * float(grad.double().norm())


@pytest.mark.parametrize("dtype", DTYPES)
def test_another_stream_and_graph(sgemm_lib, dtype):
    sg = sgemm_lib
    x, w, labels, dloss = inputs(300, 1001, 265, dtype, seed=13)

    def step(stream=None):
        loss, lse = sg.cross_entropy(x, w, labels, stream=stream)
        return (loss, lse, *sg.cross_entropy_backward(dloss, x, w, labels, lse, stream=stream))

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
        other = inputs(40, 3000, 520, dtype, seed=14)
        sg.cross_entropy(other[0], other[1], other[2])  # a call of other sizes between replays
        for _ in range(3):
            for t in got:
                t.zero_()
            graph.replay()
        s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sg.sgemm_device_status() == sg.SGEMM_OK


def test_offsets_past_32_bits(sgemm_lib):
    """Rows of x, w, dx and dw more than 2^31 values from the first."""
    sg = sgemm_lib
    T, V, D, pitch = 9, 10, 64, 1 << 28
    x, w, labels, dloss = inputs(T, V, D, ignored=0.0, seed=15)
    loss, lse = sg.cross_entropy(x, w, labels)
    dx, dw = sg.cross_entropy_backward(dloss, x, w, labels, lse)

    def far(t):
        buf = torch.empty(t.shape[0] * pitch, dtype=t.dtype, device="cuda").view(t.shape[0], pitch)[:, :t.shape[1]]
        buf.copy_(t)
        return buf

    fx, fw = far(x), far(w)
    floss, flse = sg.cross_entropy(fx, fw, labels)
    assert torch.equal(floss, loss) and torch.equal(flse, lse)
    ox, ow = far(torch.zeros_like(x)), far(torch.zeros_like(w))
    sg.sgemm_cross_entropy_backward("bf16", "T", T, V, D, dloss, 1, fx, pitch, fw, pitch, labels, lse, ox, pitch, ow, pitch)
    assert torch.equal(ox, dx) and torch.equal(ow, dw)


@pytest.mark.parametrize("transw", ["T", "N"])
def test_a_vocabulary_of_2_to_the_28(sgemm_lib, transw):
    """Weights of more than 2^31 values, in both storages, their gradient in three pieces of the vocabulary."""
    sg = sgemm_lib
    T, V, D = 3, (1 << 28) + 5, 8
    x = normal(1, T, D)
    w = torch.empty((V, D) if transw == "T" else (D, (V + 7) // 8 * 8), dtype=x.dtype, device="cuda").normal_(0.0, 0.5)
    w = w if transw == "T" else w[:, :V]
    labels = torch.tensor([0, V - 1, V // 2], device="cuda")
    loss, lse = sg.cross_entropy(x, w, labels, transw=transw)
    wt = w if transw == "T" else w.t()
    z = torch.empty(T, V, device="cuda")  # in pieces: 64 bits of all of it at once are not needed
    total = torch.zeros(T, dtype=torch.float64, device="cuda")
    step = 1 << 26
    for v in range(0, V, step):
        part = x.double() @ wt[v:v + step].double().t()
        total += part.exp().sum(1)
        z[:, v:v + step] = part.float()
    want = total.log()
    # |z| <= 8 * 12: the terms' errors 8 * ACC * 12, the sums' as in training_case.py
    assert float((lse.double() - want).abs().max()) < 2e-3
    at = torch.stack([z[t, labels[t]] for t in range(T)]).double()
    assert float((loss.double() - (want - at)).abs().max()) < 2e-3
    d = torch.full((), 1.0, device="cuda").expand(T)
    dx, dw = sg.cross_entropy_backward(d, x, w, labels, lse, transw=transw)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    dwt = dw if transw == "T" else dw.t()
    rdx = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    for v in range(0, V, step):
        dz = (z[:, v:v + step].double() - want[:, None]).exp()
        for t in range(T):
            if v <= int(labels[t]) < v + step:
                dz[t, int(labels[t]) - v] -= 1.0
        rdx += dz @ wt[v:v + step].double()
        ref = dz.t() @ x.double()
        bound = 0.02 * (dz.abs().t() @ x.double().abs()) + 1e-30
        assert bool(((dwt[v:v + step].double() - ref).abs() <= bound).all()), v
    # dz is rounded by 2^-9 of itself, and each of dx's terms with it; sum of |dz| is 2 per token, |w| < 4
    assert float((dx.double() - rdx).abs().max()) < 2.0 ** -8 * 2 * 4


def test_gradient_of_many_tokens_with_their_own_dloss(sgemm_lib):
    x, w, labels, dloss = inputs(20000, 100, 64, seed=17)
    check(sgemm_lib, x, w, labels, dloss * 20000)
