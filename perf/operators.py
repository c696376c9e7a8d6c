"""The feed-forward operators of a language model on 16-bit values, and the sizes they are
measured at: the linear layer with bias, activation and residual in its epilogue, that layer's
gradients, and a whole mixture-of-experts layer for a few tokens.

``own`` false computes them in plain torch, in 32 bits with one rounding at the end; ``own``
true calls this framework's entry points on the same tensors.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # One generated token through a feed-forward up-projection: the weights' bytes decide.
        dict(name="linear-token", op="linear", M=1, N=14336, K=4096, dtype="bf16", act="silu",
             transw="T", bias=True, residual=False, pre=False, pad=0),
        # A small layer for a handful of tokens: the call's latency decides.
        dict(name="linear-small", op="linear", M=8, N=512, K=512, dtype="f16", act="relu",
             transw="N", bias=True, residual=False, pre=False, pad=0),
        # A decoding batch through a layer of odd width, whose rows no 16-byte copy can read.
        dict(name="linear-batch-odd", op="linear", M=13, N=3001, K=1537, dtype="bf16",
             act="gelu", transw="T", bias=True, residual=True, pre=False, pad=0),
        # A short prompt through the query, key and value projection.
        dict(name="linear-prompt", op="linear", M=512, N=12288, K=4096, dtype="bf16",
             act="none", transw="T", bias=True, residual=False, pre=False, pad=0),
        # The repository's ragged edge shape, in training (the pre-activation is kept).
        dict(name="linear-ragged", op="linear", M=4095, N=3001, K=1537, dtype="f16",
             act="gelu_tanh", transw="N", bias=True, residual=True, pre=True, pad=3),
        # A training batch through the up-projection, the pre-activation kept for the gradient.
        dict(name="linear-train", op="linear", M=16384, N=14336, K=4096, dtype="bf16",
             act="gelu", transw="T", bias=True, residual=False, pre=True, pad=0),
        # Gradients of a small layer: launches and tails decide.
        dict(name="backward-small", op="backward", M=256, N=1024, K=1024, dtype="bf16",
             act="relu", transw="T", pad=0),
        # Gradients at the ragged edge shape.
        dict(name="backward-ragged", op="backward", M=4095, N=3001, K=1537, dtype="f16",
             act="gelu_tanh", transw="N", pad=3),
        # Gradients of the training batch's up-projection.
        dict(name="backward-train", op="backward", M=16384, N=14336, K=4096, dtype="bf16",
             act="gelu", transw="T", pad=0),
        # One generated token through two of eight large experts.
        dict(name="moe-token", op="moe", T=1, E=8, k=2, D=4096, F=14336, dtype="bf16",
             act="silu", gated=True, renormalize=True, residual=True, masked=False),
        # A decoding batch through many small experts, some slots of the batch idle.
        dict(name="moe-batch", op="moe", T=32, E=64, k=8, D=2048, F=1024, dtype="f16",
             act="silu", gated=True, renormalize=False, residual=True, masked=True),
        # A few tokens through odd-sized experts without a gate.
        dict(name="moe-odd", op="moe", T=7, E=4, k=1, D=1537, F=3001, dtype="bf16",
             act="gelu", gated=False, renormalize=True, residual=False, masked=False),
    ]


def _size(rng, low, high):
    """Log-uniform; half of the sizes multiples of 64, a third of 8, a sixth any."""
    v = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    step = rng.choice((64, 64, 64, 8, 8, 1))
    return max(low, min(high, (v + step // 2) // step * step))


def draw(rng):
    op = rng.choice(("linear", "backward", "moe"))
    dtype = rng.choice(("bf16", "f16"))
    act = rng.choice(ACTS)
    if op == "moe":
        while True:
            c = dict(op=op, T=int(round(math.exp(rng.uniform(0, math.log(64))))),
                     E=rng.choice((4, 8, 16, 60, 64, 128)), k=rng.choice((1, 2, 4, 6, 8)),
                     D=_size(rng, 64, 4096), F=_size(rng, 64, 14336), dtype=dtype,
                     act=rng.choice(("silu", "gelu_tanh", "relu")), gated=rng.random() < 0.75,
                     renormalize=rng.random() < 0.5, residual=rng.random() < 0.5,
                     masked=rng.random() < 0.25)
            if c["k"] <= c["E"] and c["E"] * c["D"] * c["F"] <= 8 * 4096 * 14336:
                return c
    while True:
        low = 1 if op == "linear" else 64
        M = int(round(math.exp(rng.uniform(math.log(low), math.log(16384)))))
        c = dict(op=op, M=M, N=_size(rng, 64, 14336), K=_size(rng, 64, 14336), dtype=dtype, act=act,
                 transw=rng.choice(("T", "T", "N")), pad=rng.choice((0, 0, 0, 8, 8, 5)))
        if op == "linear":
            c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5, pre=rng.random() < 0.5)
        if c["M"] * c["N"] * c["K"] <= 16384 * 14336 * 4096:
            return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _matrix(g, rows, cols, dtype, scale=1.0, pad=0):
    """rows x cols in rows of cols + pad values: a part of a wider buffer where pad > 0."""
    return _normal(g, (rows, cols + pad), dtype, scale)[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    if case["op"] == "moe":
        T, E, D, F = case["T"], case["E"], case["D"], case["F"]
        s = dict(case=case, x=_normal(g, (T, D), dt),
                 router=_normal(g, (E, D), dt, 1.5 / math.sqrt(D)),
                 gate=_normal(g, (E, F, D), dt, 1 / math.sqrt(D)) if case["gated"] else None,
                 up=_normal(g, (E, F, D), dt, 1 / math.sqrt(D)),
                 down=_normal(g, (E, D, F), dt, 1 / math.sqrt(F)),
                 residual=_normal(g, (T, D), dt) if case["residual"] else None, active=None)
        if case["masked"]:
            s["active"] = torch.rand(T, generator=g, device="cuda") < 0.75
        return s
    M, N, K, pad = case["M"], case["N"], case["K"], case["pad"]
    s = dict(case=case, x=_matrix(g, M, K, dt, 1.0, pad))
    shape = (N, K) if case["transw"] == "T" else (K, N)
    s["w"] = _matrix(g, *shape, dt, 1 / math.sqrt(K))
    if case["op"] == "linear":
        s["bias"] = _normal(g, (N,), dt, 0.5) if case["bias"] else None
        s["residual"] = _matrix(g, M, N, dt, 1.0, pad) if case["residual"] else None
    else:
        s["pre"] = _matrix(g, M, N, dt, 1.0, pad) if case["act"] != "none" else None
        s["dy"] = _matrix(g, M, N, dt, 0.05, pad)
    return s


# ---- the plain forms -------------------------------------------------------------------------

def _act(z, act):
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return z


def _act_grad(z, dy, act):
    """dy * act'(z)."""
    if act == "relu":
        return torch.where(z <= 0, torch.zeros_like(dy), dy)
    if act == "gelu":
        return dy * (0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
                     + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return dy * (0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z))
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return dy * p * (1 + z * (1 - p))
    return dy


def _plain_linear(s):
    case, dt = s["case"], s["x"].dtype
    w = s["w"].float()
    z = s["x"].float() @ (w.t() if case["transw"] == "T" else w)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return (y.to(dt), z.to(dt)) if case["pre"] else (y.to(dt),)


def _plain_backward(s):
    case, dt = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = _act_grad(s["pre"].float(), dz, case["act"])
    w, x = s["w"].float(), s["x"].float()
    if case["transw"] == "T":
        dx, dw = dz @ w, dz.t() @ x
    else:
        dx, dw = dz @ w.t(), x.t() @ dz
    return dx.to(dt), dw.to(dt), dz.sum(0)


def _plain_moe(s):
    """Every expert for every token, weighted by zero where the router left it out."""
    case, x, dt = s["case"], s["x"].float(), s["x"].dtype
    T, E, k = case["T"], case["E"], case["k"]
    logits = x @ s["router"].float().t()
    order = torch.sort(logits, dim=1, descending=True, stable=True)
    index = order.indices[:, :k]
    p = torch.exp(order.values - order.values[:, :1])
    p = p[:, :k] / (p[:, :k] if case["renormalize"] else p).sum(1, keepdim=True)
    if s["active"] is not None:
        on = s["active"][:, None]
        index = torch.where(on, index, torch.full_like(index, -1))
        p = torch.where(on, p, torch.zeros_like(p))
    share = torch.zeros(T, E + 1, device=x.device)
    share = share.scatter(1, torch.where(index < 0, torch.full_like(index, E), index), p)[:, :E]
    u = x @ s["up"].float().transpose(1, 2)  # E x T x F
    if s["gate"] is not None:
        u = u * _act(x @ s["gate"].float().transpose(1, 2), case["act"])
    else:
        u = _act(u, case["act"])
    y = ((u @ s["down"].float().transpose(1, 2)) * share.t()[:, :, None]).sum(0)
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt), index.to(torch.int32), p


def _own(s):
    import dense_fp32_gemm_08_gb300 as sg
    case = s["case"]
    if case["op"] == "linear":
        out = sg.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"],
                        transw=case["transw"], save_pre=case["pre"])
        return out if case["pre"] else (out,)
    if case["op"] == "backward":
        return sg.linear_backward(s["dy"], s["x"], s["w"], pre=s["pre"], act=case["act"],
                                  transw=case["transw"])
    return sg.moe(s["x"], s["router"], s["gate"], s["up"], s["down"], case["k"], act=case["act"],
                  renormalize=case["renormalize"], active=s["active"], residual=s["residual"])


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return {"linear": _plain_linear, "backward": _plain_backward, "moe": _plain_moe}[op](state)


def work(case):
    if case["op"] == "moe":
        T, E, k, D, F = (case[n] for n in ("T", "E", "k", "D", "F"))
        tokens = T * (0.75 if case["masked"] else 1.0)
        mats = 3 if case["gated"] else 2
        experts = E * (1 - (1 - k / E) ** tokens)  # expected number that some token chose
        return {"bytes": 2 * (experts * mats * D * F + E * D + T * D * (3 if case["residual"] else 2))
                + 8 * T * k + (T if case["masked"] else 0),
                "flops": 2 * tokens * (k * mats * D * F + E * D)}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "linear":
        return {"bytes": 2 * (M * K + N * K + M * N * (1 + case["residual"] + case["pre"])
                              + N * case["bias"]), "flops": 2 * M * N * K}
    return {"bytes": 2 * (M * N * (1 + (case["act"] != "none")) + 2 * M * K + 2 * N * K) + 4 * N,
            "flops": 4 * M * N * K}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _exact_act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def exact(case, seed):
    s = prepare(case, seed)

    def wide(t):
        return t.double()

    if case["op"] == "linear":
        w = wide(s["w"]) if case["transw"] == "N" else wide(s["w"]).T
        z = torch.mm(wide(s["x"]), w)
        del w
        if s["bias"] is not None:
            z += wide(s["bias"])
        y = _exact_act(z, case["act"])
        if s["residual"] is not None:
            y = y + wide(s["residual"])
        return (y, z) if case["pre"] else (y,)
    if case["op"] == "backward":
        dy = wide(s["dy"])
        if s["pre"] is not None:  # the slope by torch's own differentiation, in 64 bits
            z = wide(s["pre"]).requires_grad_()
            if case["act"] == "relu":
                dy = dy * (z.detach() > 0)
            else:
                dy, = torch.autograd.grad(_exact_act(z, case["act"]), z, dy)
        w = wide(s["w"]) if case["transw"] == "N" else wide(s["w"]).T
        dx = torch.mm(dy, w.T)
        dw = torch.mm(wide(s["x"]).T, dy)
        return dx, dw if case["transw"] == "N" else dw.T.contiguous(), dy.sum(dim=0)
    x, T, k = wide(s["x"]), case["T"], case["k"]
    score = torch.mm(x, wide(s["router"]).T)
    chance = torch.softmax(score, dim=1)
    y = torch.zeros_like(x) if s["residual"] is None else wide(s["residual"])
    weight = torch.zeros(T, k, dtype=torch.float64, device=x.device)
    users = {}
    for t in range(T):
        if s["active"] is not None and not bool(s["active"][t]):
            continue
        row = score[t].tolist()
        best = sorted(range(case["E"]), key=lambda e: (-row[e], e))[:k]
        c = chance[t, best]
        weight[t] = c / c.sum() if case["renormalize"] else c
        for j, e in enumerate(best):
            users.setdefault(e, []).append((t, j))
    for e, pairs in users.items():
        at = torch.tensor([t for t, _ in pairs], device=x.device)
        h = torch.mm(x[at], wide(s["up"][e]).T)
        if s["gate"] is not None:
            h = h * _exact_act(torch.mm(x[at], wide(s["gate"][e]).T), case["act"])
        else:
            h = _exact_act(h, case["act"])
        o = torch.mm(h, wide(s["down"][e]).T)
        y[at] += o * torch.stack([weight[t, j] for t, j in pairs])[:, None]
    return y, None, weight
