"""The layer operators called from several host threads: results equal those of one thread, bit for
bit (a call's sums have a fixed order, so any difference is a workspace that two calls shared)."""
from __future__ import annotations

import math
import threading

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()


def linear_inputs(seed, M, N, K):
    return normal(seed, M, K), normal(seed + 1, N, K, scale=1 / math.sqrt(K)), normal(seed + 2, M, N)


def run_together(jobs):
    """Every job in a thread of its own, all started at once; their exceptions are raised here."""
    gate, errors = threading.Barrier(len(jobs)), []

    def body(job):
        try:
            torch.cuda.set_device(0)
            gate.wait(timeout=60)
            job()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(job,)) for job in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


# Odd widths: every call repacks its operands into the stream's workspace before its product. The
# sizes go up and down, so that the workspaces grow while the other thread's calls are queued.
FORWARD = [(13, 301, 257), (300, 515, 771), (70, 1201, 1033), (13, 301, 257), (513, 2049, 1025)]
BACKWARD = [(9, 129, 67), (200, 303, 515), (700, 1025, 263), (40, 77, 901), (1100, 903, 1201)]


def test_two_threads_on_one_stream(sgemm_lib):
    sg = sgemm_lib
    forward = [linear_inputs(10 * i, *size) for i, size in enumerate(FORWARD)]
    backward = [(*linear_inputs(1000 + 10 * i, *size)[:2], normal(1005 + 10 * i, *size[:2]),
                 normal(1006 + 10 * i, *size[:2])) for i, size in enumerate(BACKWARD)]

    def linear(i):
        x, w, r = forward[i]
        return (sg.linear(x, w, act="silu", residual=r),)

    def gradients(i):
        x, w, pre, dy = backward[i]
        return sg.linear_backward(dy, x, w, pre=pre, act="silu")

    want_linear = [linear(i) for i in range(len(forward))]
    want_gradients = [gradients(i) for i in range(len(backward))]
    torch.cuda.synchronize()
    sg.sgemm_release_workspace()
    got_linear, got_gradients = [], []

    def calls(fn, n, out):
        def job():
            for k in range(100):
                out.append((k % n, fn(k % n)))
        return job

    def release():  # another thread may free the workspaces at any time
        for _ in range(10):
            sg.sgemm_release_workspace()

    run_together([calls(linear, len(forward), got_linear), calls(gradients, len(backward), got_gradients), release])
    torch.cuda.synchronize()
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    for got, want in ((got_linear, want_linear), (got_gradients, want_gradients)):
        assert len(got) == 100
        for i, tensors in got:
            assert all(torch.equal(a, b) for a, b in zip(tensors, want[i])), i


def test_experts_beside_linear_on_one_stream(sgemm_lib):
    sg = sgemm_lib
    T, E, D, F = 5, 6, 264, 328
    x, router = normal(1, T, D), normal(2, E, D, scale=0.1)
    gate, up = normal(3, E, F, D, scale=0.06), normal(4, E, F, D, scale=0.06)
    down = normal(5, E, D, F, scale=0.06)
    xl, w, _ = linear_inputs(7, 30, 333, 265)
    want_moe, want_linear = sg.moe(x, router, gate, up, down, 2), sg.linear(xl, w)
    got_moe, got_linear = [], []
    run_together([lambda: got_moe.extend(sg.moe(x, router, gate, up, down, 2) for _ in range(100)),
                  lambda: got_linear.extend(sg.linear(xl, w) for _ in range(100))])
    torch.cuda.synchronize()
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert all(torch.equal(a, b) for got in got_moe for a, b in zip(got, want_moe))
    assert all(torch.equal(got, want_linear) for got in got_linear)


def test_each_threads_default_stream_has_its_own_workspaces(sgemm_lib):
    """cudaStreamPerThread is one handle for a different stream in every thread."""
    sg = sgemm_lib
    per_thread = 2  # cudaStreamPerThread
    M, N, K = 260, 264, 4096  # cut along k: pieces and arrival counters in the workspace
    xs = [normal(i, M, K) for i in range(3)]
    w = normal(9, N, K, scale=1 / 64)
    want = [sg.linear(x, w, act="gelu") for x in xs]
    outs = [[torch.zeros_like(want[0]) for _ in range(40)] for _ in xs]
    torch.cuda.synchronize()

    def calls(i):
        def job():
            for out in outs[i]:
                sg.sgemm_linear("bf16", "T", M, N, K, xs[i], K, w, K, None, "gelu", None, 0, out, N,
                                stream=per_thread)
        return job

    run_together([calls(i) for i in range(len(xs))])
    torch.cuda.synchronize()
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    for i, group in enumerate(outs):
        assert all(torch.equal(out, want[i]) for out in group), i
