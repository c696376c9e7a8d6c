"""Graphs of the layer operators' calls: replays after larger calls on the same stream, and captures
that would have to allocate."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def linear_case(seed, M, N, K):
    """A call with an output of its own: odd sizes are repacked, long k with few tiles is cut."""
    x, w, r = normal(seed, M, K), normal(seed + 1, N, K, scale=1 / math.sqrt(K)), normal(seed + 2, M, N)
    out = torch.zeros(M, N, dtype=x.dtype, device="cuda")
    return out, lambda sg: sg.linear(x, w, act="silu", residual=r, out=out)


def gradient_case(seed, M, N, K):
    x, w = normal(seed, M, K), normal(seed + 1, N, K, scale=1 / math.sqrt(K))
    pre, dy = normal(seed + 2, M, N), normal(seed + 3, M, N)
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    db = torch.zeros(N, device="cuda")

    def call(sg):
        sg.sgemm_linear_backward("bf16", "T", M, N, K, dy, N, pre, N, "silu", x, K, w, K, dx, K, dw, K, db)
    return (dx, dw, db), call


def moe_case(seed, T, E, D, F, k):
    x, router = normal(seed, T, D), normal(seed + 1, E, D, scale=0.1)
    gate, up = normal(seed + 2, E, F, D, scale=0.06), normal(seed + 3, E, F, D, scale=0.06)
    down = normal(seed + 4, E, D, F, scale=0.06)
    out = torch.zeros_like(x)
    return out, lambda sg: sg.moe(x, router, gate, up, down, k, residual=x, out=out)


SMALL_AND_LARGE = {
    "linear-repacked": (lambda: linear_case(1, 30, 301, 257), lambda: linear_case(5, 600, 1301, 1257)),
    "linear-cut": (lambda: linear_case(1, 260, 264, 4096), lambda: linear_case(5, 1024, 1024, 8192)),
    "gradients": (lambda: gradient_case(1, 700, 130, 70), lambda: gradient_case(5, 4000, 1304, 520)),
    "experts": (lambda: moe_case(1, 4, 8, 256, 320, 2), lambda: moe_case(9, 60, 32, 1024, 1152, 4)),
    "experts-unaligned": (lambda: moe_case(1, 3, 4, 129, 131, 2), lambda: moe_case(9, 20, 8, 257, 1031, 4)),
}


def tensors(out):
    return out if isinstance(out, tuple) else (out,)


@pytest.mark.parametrize("name", SMALL_AND_LARGE)
def test_replay_after_a_larger_call(sgemm_lib, name):
    sg = sgemm_lib
    small, large = (make() for make in SMALL_AND_LARGE[name])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        small[1](sg)
        torch.cuda.synchronize()
        want = [t.clone() for t in tensors(small[0])]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            small[1](sg)
        large[1](sg)  # its workspaces outgrow the captured call's
        torch.cuda.synchronize()
        large_want = [t.clone() for t in tensors(large[0])]
        fill = [torch.full((1 << 20,), math.nan, device="cuda") for _ in range(32)]  # would take freed memory
        for _ in range(3):
            for t in tensors(small[0]):
                t.fill_(7.0)
            graph.replay()
            large[1](sg)
        torch.cuda.synchronize()
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert all(torch.equal(a, b) for a, b in zip(tensors(small[0]), want))
    assert all(torch.equal(a, b) for a, b in zip(tensors(large[0]), large_want))
    assert all(bool(torch.isnan(f).all()) for f in fill)


def test_a_capture_that_would_allocate_is_refused(sgemm_lib):
    sg = sgemm_lib
    small, large = linear_case(1, 30, 301, 257), linear_case(5, 1600, 3301, 1257)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        sg.sgemm_release_workspace()
        small[1](sg)
        torch.cuda.synchronize()
        want = small[0].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            with pytest.raises(sg.SgemmError, match="before the capture"):
                large[1](sg)
            small[1](sg)  # the capture goes on
        small[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(small[0], want)
        large[1](sg)  # and outside it the larger call runs
        torch.cuda.synchronize()
    assert bool(torch.isfinite(large[0].float()).all()) and bool(large[0].any())
    assert sg.sgemm_device_status() == sg.SGEMM_OK
