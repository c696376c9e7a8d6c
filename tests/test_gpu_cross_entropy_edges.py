"""GPU parity of the head's cross entropy where its values are not finite or its labels all but certain."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import training_case as case  # noqa: E402
from layer_case import worst  # noqa: E402

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]
# Few tokens, more of them on the streaming product, and the pair product (more than 128 tiles of 64 x 128).
TOKENS_AND_ENTRIES = [(3, 300), (140, 700), (700, 3001)]


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def inputs(T, V, D, dtype=torch.bfloat16, transw="T", seed=0):
    x = normal(seed + 1, T, D, dtype=dtype)
    w = normal(seed + 2, V, D, dtype=dtype, scale=1.5 / math.sqrt(D))
    g = torch.Generator(device="cuda").manual_seed(seed)
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    return x, w if transw == "T" else w.t().contiguous(), labels


@pytest.mark.parametrize("T,V", TOKENS_AND_ENTRIES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_token_with_a_nan_has_nan_lse(sgemm_lib, dtype, T, V):
    """Every logit of the token is NaN: lse too, whether or not the token counts, and no other token's."""
    sg = sgemm_lib
    x, w, labels = inputs(T, V, 72, dtype, seed=T)
    want_loss, want_lse = sg.cross_entropy(x, w, labels)
    x[0, 3], x[2, 70] = math.nan, math.nan
    labels[2] = -100
    loss, lse = sg.cross_entropy(x, w, labels)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert bool(torch.isnan(lse[0])) and bool(torch.isnan(lse[2]))
    assert bool(torch.isnan(loss[0])) and float(loss[2]) == 0.0
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[0] = keep[2] = False
    assert torch.equal(lse[keep], want_lse[keep]) and torch.equal(loss[keep], want_loss[keep])
    alone = torch.empty_like(lse)
    sg.sgemm_cross_entropy("bf16" if dtype is torch.bfloat16 else "f16", "T", T, V, 72, x, 72, w, 72, labels, None, alone)
    assert torch.equal(alone.isnan(), lse.isnan()) and torch.equal(alone[keep], lse[keep])


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("T,V", TOKENS_AND_ENTRIES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
def test_one_dloss_for_all_that_is_not_finite(sgemm_lib, T, V, dtype, transw, value):
    """dz is 0 for tokens that do not count, whatever dloss: their dX, and dW where none counts, as a mean
    over no token has it. Given once for all tokens or for each, the results are the same."""
    sg = sgemm_lib
    x, w, labels = inputs(T, V, 72, dtype, transw, seed=T)
    labels[::2] = -100
    _, lse = sg.cross_entropy(x, w, labels, transw=transw)
    once = torch.full((), value, device="cuda").expand(T)
    dx, dw = sg.cross_entropy_backward(once, x, w, labels, lse, transw=transw)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert not dx[::2].any()
    assert not bool(torch.isfinite(dx[1::2]).any()) and not bool(torch.isfinite(dw).all())
    each = sg.cross_entropy_backward(once.contiguous(), x, w, labels, lse, transw=transw)
    assert same(dx, each[0]) and same(dw, each[1])
    labels[:] = V
    dx, dw = sg.cross_entropy_backward(once, x, w, labels, lse, transw=transw)
    assert not dx.any() and not dw.any()


def test_a_mean_over_no_token(sgemm_lib):
    """The gradient of sum / count where no token counts: dloss is 1 / 0 for all of them."""
    sg = sgemm_lib
    x, w, labels = inputs(20, 300, 64)
    labels[:] = -100
    loss, lse = sg.cross_entropy(x, w, labels)
    loss.requires_grad_()
    (dloss,) = torch.autograd.grad(loss.sum() / (labels >= 0).sum(), loss)
    assert bool(torch.isinf(dloss).all()) and dloss.stride(0) == 0
    dx, dw = sg.cross_entropy_backward(dloss, x, w, labels, lse)
    assert not dx.any() and not dw.any()


def fp32_step(v):
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1e-30))) - 23)


@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,V,D", [(7, 56, 704), (7, 520, 704), (64, 4000, 1000), (300, 512, 1537), (300, 4000, 704),
                                   (2304, 520, 704), (8256, 56, 704), (40000, 56, 712),
                                   (300, 4000, 4104), (40000, 9001, 72)])
def test_certain_labels_of_any_vocabulary(sgemm_lib, dtype, transw, T, V, D):
    """1 - p at the labels is about 10^-4 in each vocabulary, on either product and with tokens or entries in pieces, and
    the gradient no larger, so that the label's logit's own error shows in it. That logit is held to one step of fp32 (its
    products are added up with their roundings kept); times p < 1 it passes to dX through the label's row of W, with two
    steps of 1 - p from expm1f. Besides, 2^-14 of each other p (logits below 8 lose up to a step, 2^-21, per 16
    products, in two runs of 1024 at most, or 2^-23 at less than 2 in five of them); a rounding of each dz to 16 bits
    (and half of a subnormal step over 2^14 in half); and dX's own sum and rounding. z - lse is exact: they are within
    a factor 2 of each other."""
    sg = sgemm_lib
    u = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[dtype] * 1.001
    tiny = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}[dtype]
    g = torch.Generator(device="cuda").manual_seed(T)
    w = normal(1, V, D, dtype=dtype, scale=1.28 / math.sqrt(D))
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    sure = 8.5 + math.log(V / 56) / 1.28 ** 2  # the label's logit leaves the others' sum as far behind
    x = (normal(2, T, D, dtype=dtype).float() + sure * w[labels].float()).to(dtype)
    given = w if transw == "T" else w.t().contiguous()
    ones = torch.full((), 1.0, device="cuda").expand(T)
    z = x.double() @ w.double().t()
    exact = torch.logsumexp(z, 1).float()
    loss, own = sg.cross_entropy(x, given, labels, transw=transw)
    zl = z.gather(1, labels[:, None])
    step = fp32_step(zl[:, 0])
    # The loss: a step of the label's logit, 2^-14 of the others' share, lse in fp32 from m ln 2 (two roundings, m's and
    # the product's, of 2^-24 each) and its sum's roundings (64 + parts' joins), all of them times lse < 32 or p < 1
    rest = -torch.expm1(zl[:, 0] - torch.logsumexp(z, 1))
    assert bool(((loss.double() - (torch.logsumexp(z, 1) - zl[:, 0])).abs() <= 2 * step + 2.0 ** -14 * rest
                 + (4 * exact.abs() + 64 + V / 256 + 16) * 2.0 ** -24 + 2.0 ** -22).all())
    length = w.double().norm(dim=1)
    for lse in (exact, own):
        dx, _ = sg.cross_entropy_backward(ones, x, given, labels, lse, transw=transw)
        assert sg.sgemm_device_status() == sg.SGEMM_OK
        gap = z - lse.double()[:, None]
        dz = torch.exp(gap)
        dz.scatter_(1, labels[:, None], torch.expm1(gap.gather(1, labels[:, None])))
        ref = dz @ w.double()
        at = dz.gather(1, labels[:, None])[:, 0].abs()
        off = (2.0 ** -14 + u) * (dz.abs() @ length) + (step + 2.0 ** -22 * at) * length[labels]
        small = 0.0 if dtype is torch.bfloat16 else 2.0 ** -25 * 2.0 ** -14
        off += small * length.sum() + 1e-5 * (dz.abs() @ w.double().abs()).norm(dim=1)
        off += u * ref.norm(dim=1) + tiny * math.sqrt(D)
        ratio = (dx.double() - ref).norm(dim=1) / off
        assert bool((ratio <= 1.0).all()), float(ratio.max())


def test_logits_are_summed_in_runs(sgemm_lib):
    """The pair product's accumulators lose up to a step of fp32 per 16 products, always towards zero (the tensor
    cores cut). From zero in each run of 1024 products, and half a step for each run added, that bounds how far lse is
    below its value where all products are positive; one accumulator for all 4104 would lose half of its own bound on
    average, which is more. (In lse an error of every logit counts once, since the probabilities add up to 1; the
    exponentials, their sums and lse's rounding are as in training_case.py.)"""
    sg, (T, V, D) = sgemm_lib, (300, 3500, 4104)
    x = normal(1, T, D).abs()
    w = (normal(2, V, D).abs().float() * (12.0 / (D * 2 / math.pi))).bfloat16()
    labels = torch.full((T,), -100, device="cuda")
    _, lse = sg.cross_entropy(x, w, labels)
    xd, wd = x.double(), w.double()

    def lost(run):
        total, all_lost = torch.zeros(T, V, dtype=torch.float64, device="cuda"), torch.zeros(T, V, device="cuda")
        for r in range(0, D, run):
            part = torch.zeros_like(total)
            for k in range(r, min(r + run, D), 16):
                end = min(k + 16, r + run, D)
                part += xd[:, k:end] @ wd[:, k:end].t()
                all_lost += fp32_step(part)
            total += part
            if r > 0:
                all_lost += fp32_step(total) / 2
        return total, all_lost.double()

    z, bound = lost(1024)
    want = torch.logsumexp(z, 1)
    bound = (torch.softmax(z, 1) * bound).sum(1).mean()
    rest = ((64 + V / 64 / 32 * 8 + 16) * 2.0 ** -24 + 2.0 ** -22 * want.abs()).mean()
    one = (torch.softmax(z, 1) * lost(D)[1]).sum(1).mean() / 2
    assert float(one) > float(bound + rest)
    assert float((want - lse.double()).mean()) <= float(bound + rest)
    assert float((lse.double() - want).mean()) <= float(rest)


def certain(T, V, D, dtype, transw, seed=0):
    """Half of the labels all but certain, some that do not count."""
    w = normal(seed + 1, V, D, dtype=dtype, scale=1.28 / math.sqrt(D))
    g = torch.Generator(device="cuda").manual_seed(seed)
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    sure = (8.5 + math.log(V / 56) / 1.28 ** 2) * (torch.arange(T, device="cuda") % 2)[:, None]
    x = (normal(seed + 2, T, D, dtype=dtype).float() + sure * w[labels].float()).to(dtype)
    labels[::5] = -100
    dloss = torch.randn(T, generator=g, device="cuda") / T
    return x, w if transw == "T" else w.t().contiguous(), labels, dloss


def wider(t, pad, offset=0):
    rows, cols = t.shape
    buf = torch.full((rows * (cols + pad) + offset,), math.nan, dtype=t.dtype, device="cuda")
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(t)
    return view


def both(sg, x, w, labels, dloss, transw, stream=None):
    loss, lse = sg.cross_entropy(x, w, labels, transw=transw, stream=stream)
    return (loss, lse, *sg.cross_entropy_backward(dloss, x, w, labels, lse, transw=transw, stream=stream))


@pytest.mark.parametrize("T,V,D", [(5, 77, 129), (40, 700, 265), (700, 3001, 200), (8300, 60, 71)])
@pytest.mark.parametrize("transw", ["T", "N"])
@pytest.mark.parametrize("dtype", DTYPES)
def test_certain_labels_in_other_layouts(sgemm_lib, dtype, transw, T, V, D):
    """The same values in wider or unaligned rows, weights of the tokens in a strided column: the same results to the
    bit; and those within the tolerances of the definitions."""
    sg = sgemm_lib
    x, w, labels, dloss = certain(T, V, D, dtype, transw, seed=T)
    want = both(sg, x, w, labels, dloss, transw)
    column = torch.zeros(T, 3, device="cuda")
    column[:, 1] = dloss
    for pad, offset in ((3, 0), (8, 0), (0, 1), (5, 8)):
        got = both(sg, wider(x, pad, offset), wider(w, pad, offset), labels, column[:, 1], transw)
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    loss, lse, dx, dw = want
    rloss, rlse, _, tol, ltol, _ = case.head_ref(x, w, labels, transw)
    assert worst(lse, rlse, ltol) <= 1.0 and worst(loss, rloss, tol) <= 1.0
    rdx, rdw, dxtol, dwtol = case.head_grad_ref(dloss, x, w, labels, lse, transw)
    assert worst(dx, rdx, dxtol) <= 1.0 and worst(dw, rdw, dwtol) <= 1.0
    assert not dx[::5].any()


@pytest.mark.parametrize("T,V", TOKENS_AND_ENTRIES)
def test_certain_labels_on_a_stream_and_in_a_graph(sgemm_lib, T, V):
    sg = sgemm_lib
    args = certain(T, V, 264, torch.bfloat16, "T", seed=V)
    want = both(sg, *args, "T")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = both(sg, *args, "T", stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = both(sg, *args, "T")
        for _ in range(3):
            for t in got:
                t.fill_(7.0)
            graph.replay()
        s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sg.sgemm_device_status() == sg.SGEMM_OK


@pytest.mark.parametrize("transw", ["T", "N"])
def test_one_entry_has_no_loss(sgemm_lib, transw):
    """A vocabulary of one entry: lse is its logit z, the loss and p - 1 are zero but for lse's roundings. With m = z log2 e
    rounded, the sum is 2^(z log2 e - m), off by 2^-22 (the hardware's exponential) and its rounding; its logarithm by that
    and 2^-24; m ln 2 is added in two parts, rounded to a step of z at the end, and once more with the label's logit
    (within a step too): e = 2^-21 + 3 |z| 2^-23 bounds the loss and |p - 1|, and its products the gradients."""
    sg = sgemm_lib
    for T in (1, 70, 9000):  # (the last on the pair product)
        x, w, labels = inputs(T, 1, 520, transw=transw, seed=T)
        labels[1::3] = -100
        loss, lse, dx, dw = both(sg, x, w, labels, torch.ones(T, device="cuda"), transw)
        row = w.double().reshape(-1)
        z = x.double() @ row
        e = (2.0 ** -21 + 3 * z.abs() * 2.0 ** -23) * 1.01 * (labels >= 0)
        assert bool((loss >= 0).all()) and bool((loss.double() <= e).all())
        assert bool(((lse.double() - z).abs() <= e)[labels >= 0].all())
        assert bool((dx.double().abs() <= e[:, None] * row.abs() * 1.01).all())
        assert bool((dw.double().abs().reshape(-1) <= e @ x.double().abs() * 1.01).all())
