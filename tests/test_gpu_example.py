"""The feed-forward example runs as a user would run it, trains, and serves what the plain
definitions give."""
from __future__ import annotations

import importlib.util
from pathlib import Path

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]


def _example():
    spec = importlib.util.spec_from_file_location("feed_forward", ROOT / "examples" / "feed_forward.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_training_lowers_the_loss(sgemm_lib):
    losses = _example().train()
    assert all(b < a for a, b in zip(losses, losses[1:])), losses
    assert losses[-1] < 0.9 * losses[0]


def test_gradients_match_autograd(sgemm_lib):
    """The example's block against torch's own differentiation of the same block in 64 bits, each
    gradient within 2% in norm: every value passes four roundings of 2^-8 (h, dz, its own and the
    incoming gradient's), which add up to about 1%."""
    ex = _example()
    g = torch.Generator(device="cuda").manual_seed(3)
    p = {n: (torch.randn(*s, generator=g, device="cuda") * 0.1).bfloat16().requires_grad_()
         for n, s in (("w1", (384, 256)), ("b1", (384,)), ("w2", (256, 384)), ("b2", (256,)))}
    x = torch.randn(200, 256, generator=g, device="cuda").bfloat16().requires_grad_()
    c = torch.randn(200, 256, generator=g, device="cuda").bfloat16()
    got = torch.autograd.grad(ex.block(x, p), [x, *p.values()], c)
    xd, *pd = (t.detach().double().requires_grad_() for t in (x, *p.values()))
    y = xd + torch.nn.functional.gelu(xd @ pd[0].t() + pd[1]) @ pd[2].t() + pd[3]
    want = torch.autograd.grad(y, [xd, *pd], c.double())
    for a, b in zip(got, want):
        assert a.shape == b.shape
        assert float((a.double() - b).norm() / b.norm()) < 0.02


def test_serving_step(sgemm_lib):
    y, index, weight = _example().serve()
    assert y.shape == (4, 1024) and bool(torch.isfinite(y).all())
    assert torch.allclose(weight.sum(1), torch.ones(4, device="cuda"))
    assert sgemm_lib.sgemm_device_status() == sgemm_lib.SGEMM_OK
