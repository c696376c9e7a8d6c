"""GPU parity of the head's cross entropy where its values are not finite or its labels all but certain."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

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
