"""The training operators together, as a step uses them: 8-bit checkpoints, the head's loss and the
gradients of both, from the example, on other streams, in graphs and from several threads."""
from __future__ import annotations

import importlib.util
import math
import threading
from pathlib import Path

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

ROOT = Path(__file__).resolve().parents[1]


def example():
    spec = importlib.util.spec_from_file_location("feed_forward", ROOT / "examples" / "feed_forward.py")
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def normal(seed, *shape, scale=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def test_the_example_trains(sgemm_lib):
    losses = example().train_tokens(steps=3)
    assert len(losses) == 3 and all(math.isfinite(v) for v in losses)
    assert sgemm_lib.sgemm_device_status() == sgemm_lib.SGEMM_OK


def test_gradients_of_the_example(sgemm_lib):
    """The example's loss against torch's own differentiation of it in 64 bits, each gradient within 3% in
    norm. A checkpoint's error is uniform within half a step of a / 127, a some 2.5 times the values' own
    size: 0.6% each for x, h and the pre-activation (whose slope passes on less); the 16-bit roundings of 2^-9
    and less rms at h, y, dz, the head's dz and each gradient add another 1%."""
    ex = example()
    T, D, F, V = 300, 136, 200, 515
    g = torch.Generator(device="cuda").manual_seed(3)
    shapes = (("w1", (F, D)), ("b1", (F,)), ("w2", (D, F)), ("b2", (D,)), ("head", (V, D)))
    p = {n: (torch.randn(*s, generator=g, device="cuda") * 0.1).bfloat16().requires_grad_() for n, s in shapes}
    x = torch.randn(T, D, generator=g, device="cuda").bfloat16().requires_grad_()
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    labels[::5] = -100
    got = torch.autograd.grad(ex.token_loss(x, p, labels), [x, *p.values()])
    xd, *pd = (t.detach().double().requires_grad_() for t in (x, *p.values()))
    y = xd + torch.nn.functional.gelu(xd @ pd[0].t() + pd[1]) @ pd[2].t() + pd[3]
    want = torch.autograd.grad(torch.nn.functional.cross_entropy(y @ pd[4].t(), labels), [xd, *pd])
    for a, b in zip(got, want):
        assert a.shape == b.shape
        assert float((a.double() - b).norm() / b.norm()) < 0.03


def step(sg, seed, M=300, D=264, F=520, V=1001, dtype=torch.bfloat16):
    """One forward and backward pass of two layers and the head; the call and its inputs."""
    x = normal(seed, M, D, dtype=dtype)
    w1, w2 = normal(seed + 1, F, D, scale=D ** -0.5, dtype=dtype), normal(seed + 2, D, F, scale=F ** -0.5, dtype=dtype)
    head = normal(seed + 3, V, D, scale=D ** -0.5, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    labels = torch.randint(V, (M,), generator=g, device="cuda")
    labels[::7] = -100
    dloss = torch.full((), 8.0 / M, device="cuda").expand(M)

    def call(stream=None):
        x8 = sg.checkpoint8(x, stream=stream)
        h, pre = sg.linear(x, w1, act="silu", save_pre="8bit", stream=stream)
        h8 = sg.checkpoint8(h, stream=stream)
        y = sg.linear(h, w2, residual=x, stream=stream)
        loss, lse = sg.cross_entropy(y, head, labels, stream=stream)
        dy, dhead = sg.cross_entropy_backward(dloss, y, head, labels, lse, stream=stream)
        dh, dw2, _ = sg.linear_backward(dy, h8, w2, need_db=False, stream=stream)
        dx, dw1, db1 = sg.linear_backward(dh, x8, w1, pre=pre, act="silu", stream=stream)
        return loss, lse, dhead, dw2, dx, dw1, db1

    return call


def equal(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("sizes", [dict(), dict(M=40, D=136, F=72, V=300), dict(M=33, D=129, F=65, V=77)])
def test_a_step_on_another_stream_and_in_a_graph(sgemm_lib, sizes):
    sg = sgemm_lib
    call, larger = step(sg, 1, **sizes), step(sg, 9, M=700, D=520, F=1032, V=3001)
    want = call()
    large_want = larger()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = call(s)
    s.synchronize()
    assert equal(got, want)
    with torch.cuda.stream(s):
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            got = call()
        for _ in range(2):
            assert equal(larger(), large_want)  # outgrows the captured call's workspaces
            for t in got:
                t.fill_(7.0)
            graph.replay()
        s.synchronize()
    assert equal(got, want)
    assert sg.sgemm_device_status() == sg.SGEMM_OK


def test_a_capture_that_would_allocate_is_refused(sgemm_lib):
    sg = sgemm_lib
    x, w = normal(1, 2000, 520), normal(2, 4001, 520, scale=1 / 22)
    labels = torch.zeros(2000, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        sg.sgemm_release_workspace()
        graph = torch.cuda.CUDAGraph()
        kept = torch.ones(4, device="cuda")
        with torch.cuda.graph(graph, stream=s):
            kept.add_(1.0)
            with pytest.raises(sg.SgemmError, match="before the capture"):
                sg.cross_entropy(x, w, labels)
        graph.replay()
        s.synchronize()
        loss, _ = sg.cross_entropy(x, w, labels)
        s.synchronize()
    assert bool((kept == 2.0).all()) and bool(torch.isfinite(loss).all())
    assert sg.sgemm_device_status() == sg.SGEMM_OK


def test_two_threads_on_one_stream(sgemm_lib):
    """Calls from two host threads on one stream share its workspaces, one call at a time."""
    sg = sgemm_lib
    calls = [step(sg, 1), step(sg, 5, M=90, D=136, F=300, V=2000, dtype=torch.float16)]
    want = [c() for c in calls]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        torch.cuda.set_device(0)
        for _ in range(20):
            got = calls[i]()
            torch.cuda.current_stream().synchronize()
            if not equal(got, want[i]):
                bad.append(i)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
    assert sg.sgemm_device_status() == sg.SGEMM_OK


def test_two_streams_at_once(sgemm_lib):
    """Steps queued on two streams without waiting in between: each stream has its own workspaces."""
    sg = sgemm_lib
    calls = [step(sg, 1, M=700, D=520, F=1032, V=3001), step(sg, 5, M=90, D=136, F=300, V=2000)]
    want = [c() for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    assert all(equal(g, want[i]) for i in range(2) for g in got[i])
    assert sg.sgemm_device_status() == sg.SGEMM_OK


@pytest.mark.parametrize("what", ["checkpoint", "restore", "linear", "loss", "gradient"])
def test_dropped_tensors_wait_for_the_side_stream(sgemm_lib, what):
    """The memory of a side stream's call is handed out again only when that stream is done: its inputs,
    its outputs and a checkpoint's buffer are dropped while it is still busy."""
    sg = sgemm_lib
    s = torch.cuda.Stream()
    M, N = 1024, 2048
    x, w = normal(1, M, N), normal(2, N, N, scale=N ** -0.5)
    labels = torch.arange(M, device="cuda")
    c = sg.checkpoint8(x)
    loss, lse = sg.cross_entropy(x, w, labels)
    d = torch.ones(M, device="cuda")

    def call(x, w, c, stream):
        return {"checkpoint": lambda: (sg.restore8(sg.checkpoint8(x, stream=stream), stream=stream),),
                "restore": lambda: (sg.restore8(c, stream=stream),),
                "linear": lambda: (sg.linear(x, w, act="silu", save_pre="8bit", stream=stream)[0],),
                "loss": lambda: sg.cross_entropy(x, w, labels, stream=stream),
                "gradient": lambda: sg.cross_entropy_backward(d, x, w, labels, lse, stream=stream)}[what]()

    want = call(x, w, c, None)
    call(x, w, c, s)  # the stream's workspaces exist from here on
    torch.cuda.synchronize()
    x2, w2, c2 = x.clone(), w.clone(), sg.checkpoint8(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(400_000_000)
    got = call(x2, w2, c2, s)
    del x2, w2, c2
    fill = [torch.full((M * N,), math.nan, dtype=x.dtype, device="cuda") for _ in range(4)]  # takes freed memory
    fill += [torch.full((M * N * 17 // 16,), 77, dtype=torch.int8, device="cuda") for _ in range(2)]
    s.synchronize()
    assert equal(got, want)
    del fill


def test_one_device_at_a_time(sgemm_lib):
    """Tensors that are not on the current device, or on none, are refused."""
    sg = sgemm_lib
    x, w = normal(1, 8, 16), normal(2, 8, 16)
    labels = torch.zeros(8, dtype=torch.int64)
    with pytest.raises(ValueError):
        sg.cross_entropy(x, w, labels)  # labels on the host
    with pytest.raises(ValueError):
        sg.linear_backward(x[:, :8].contiguous(), sg.Checkpoint8(torch.zeros(8, 16, dtype=torch.int8), torch.zeros(8, 1),
                                                                 torch.bfloat16), w)
