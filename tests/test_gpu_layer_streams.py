"""Calls on a stream that is not the current one: which memory their outputs get, and when the memory
of their tensors may be handed out again. (Each test looks at addresses while work is pending.)"""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROWS, WIDTH = 40, 1 << 15  # outputs of 2.5 MiB: a block of the allocator's own


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def busy():
    """Some 0.2 s of work on the current stream, far longer than the calls after it take to queue."""
    torch.cuda._sleep(400_000_000)


def linear(sg, stream):
    x, w = normal(1, ROWS, 64), normal(2, WIDTH, 64, scale=1 / 8)
    want = sg.linear(x, w)
    torch.cuda.synchronize()
    return [x, w], lambda: (sg.linear(x, w, stream=stream),), (want,)


def gradients(sg, stream):
    x, w = normal(1, ROWS, WIDTH), normal(2, 64, WIDTH, scale=1 / 181)
    dy = normal(3, ROWS, 64)
    want = sg.linear_backward(dy, x, w)
    torch.cuda.synchronize()
    return [x, w, dy], lambda: sg.linear_backward(dy, x, w, stream=stream), want


def experts(sg, stream):
    E, D, F = 2, WIDTH, 64
    x, router = normal(1, ROWS, D), normal(2, E, D, scale=0.01)
    up, down = normal(3, E, F, D, scale=1 / 181), normal(4, E, D, F, scale=1 / 8)
    want = sg.moe(x, router, None, up, down, 1)
    torch.cuda.synchronize()
    return [x, router, up, down], lambda: sg.moe(x, router, None, up, down, 1, stream=stream), want


def product(sg, stream):
    a, b = normal(1, ROWS, 64).float(), normal(2, 64, WIDTH // 2).float()
    want = sg.matmul(a, b)
    torch.cuda.synchronize()
    return [a, b], lambda: (sg.matmul(a, b, stream=stream),), (want,)


CALLS = [linear, gradients, experts, product]


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
@pytest.mark.parametrize("by_address", [False, True])
def test_outputs_do_not_take_memory_in_use(sgemm_lib, make, by_address):
    s = torch.cuda.Stream()
    _, call, want = make(sgemm_lib, s.cuda_stream if by_address else s)
    spare = [torch.empty_like(t) for t in want if t.numel() > 1 << 19]
    addresses = {t.data_ptr() for t in spare}
    assert addresses
    torch.cuda.synchronize()
    busy()
    kept = [t.clone() for t in spare]  # the current stream has yet to read them
    del spare
    got = call()
    assert not addresses & {t.data_ptr() for t in got}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert sgemm_lib.sgemm_device_status() == sgemm_lib.SGEMM_OK
    del kept


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_dropped_outputs_wait_for_both_streams(sgemm_lib, make):
    s = torch.cuda.Stream()
    _, call, want = make(sgemm_lib, s)
    call()  # the stream's workspaces exist from here on
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy()
    got = call()
    big = [(t.data_ptr(), t.shape, t.dtype) for t in got if t.numel() > 1 << 19]
    del got  # the side stream has yet to write them
    fresh = [torch.empty(shape, dtype=dtype, device="cuda") for _, shape, dtype in big]
    assert not {p for p, _, _ in big} & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    del fresh
    got = call()
    torch.cuda.current_stream().wait_stream(s)
    busy()
    kept = [t.clone() for t in got]  # the current stream has yet to read them
    big = [(t.data_ptr(), t.shape, t.dtype) for t in got if t.numel() > 1 << 19]
    del got
    with torch.cuda.stream(s):
        fresh = [torch.empty(shape, dtype=dtype, device="cuda") for _, shape, dtype in big]
    assert not {p for p, _, _ in big} & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(kept, want))


@pytest.mark.parametrize("make", CALLS, ids=lambda f: f.__name__)
def test_dropped_inputs_wait_for_the_side_stream(sgemm_lib, make):
    s = torch.cuda.Stream()
    inputs, call, want = make(sgemm_lib, s)
    call()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy()
    got = call()
    big = [(t.data_ptr(), t.shape, t.dtype) for t in inputs if t.numel() > 1 << 19]
    assert big
    inputs.clear()
    del call  # the side stream has yet to read them
    fresh = [torch.full(shape, math.nan, dtype=dtype, device="cuda") for _, shape, dtype in big]
    assert not {p for p, _, _ in big} & {t.data_ptr() for t in fresh}
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_default_stream_as_the_side_stream(sgemm_lib):
    sg = sgemm_lib
    x, w = normal(1, 8, 64), normal(2, 72, 64, scale=1 / 8)
    want = sg.linear(x, w)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for stream in (0, 1, torch.cuda.default_stream()):
            y = sg.linear(x, w, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(y, want)
    assert torch.equal(sg.linear(x, w, stream=0), want)
