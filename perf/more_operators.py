"""What a training step keeps, on 16-bit values, and the sizes it is measured at: activation
checkpoints in 8 bits, the linear layer that keeps its pre-activation in 8 bits, its gradients from
8-bit checkpoints, and the softmax cross entropy of a vocabulary head with its gradient.

``own`` false computes them in plain torch, in 32 bits with one rounding at the end; ``own``
true calls this framework's entry points on the same tensors.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BLOCK = 64  # columns that share a scale


def listed():
    return [
        # A small layer's activations, saved and restored: the calls' latency decides.
        dict(name="checkpoint-small", op="checkpoint", M=64, N=512, dtype="f16", pad=0),
        # The repository's ragged edge shape, in rows no 16-byte copy can read.
        dict(name="checkpoint-ragged", op="checkpoint", M=4095, N=3001, dtype="bf16", pad=3),
        # The hidden activations of a training batch.
        dict(name="checkpoint-train", op="checkpoint", M=16384, N=14336, dtype="bf16", pad=0),
        # A small layer's forward pass that keeps its pre-activation in 8 bits.
        dict(name="linear8-small", op="linear8", M=256, N=1024, K=1024, dtype="bf16", act="silu",
             transw="T", bias=True, residual=True, pad=0),
        # A training batch through the up-projection.
        dict(name="linear8-train", op="linear8", M=16384, N=14336, K=4096, dtype="bf16",
             act="gelu", transw="T", bias=True, residual=False, pad=0),
        # Gradients from 8-bit checkpoints at the ragged edge shape.
        dict(name="backward8-ragged", op="backward8", M=4095, N=3001, K=1537, dtype="f16",
             act="gelu_tanh", transw="N", pad=3),
        # Gradients of the training batch's up-projection from 8-bit checkpoints.
        dict(name="backward8-train", op="backward8", M=16384, N=14336, K=4096, dtype="bf16",
             act="gelu", transw="T", pad=0),
        # The log-probability of one token: the head's weights are read once.
        dict(name="loss-token", op="loss", T=1, V=32000, D=4096, dtype="bf16", transw="T",
             ignored=0.0, pad=0),
        # Scoring one odd-sized prompt, most of it not scored.
        dict(name="loss-prompt-odd", op="loss", T=777, V=30001, D=1537, dtype="f16", transw="T",
             ignored=0.6, pad=0),
        # The loss of a training batch.
        dict(name="loss-train", op="loss", T=16384, V=32000, D=4096, dtype="bf16", transw="T",
             ignored=0.1, pad=0),
        # The loss's gradient for a small vocabulary (bytes, characters): launches and tails decide.
        dict(name="loss_grad-small", op="loss_grad", T=256, V=1000, D=512, dtype="f16", transw="N",
             ignored=0.1, pad=0),
        # The loss's gradient of a training batch.
        dict(name="loss_grad-train", op="loss_grad", T=16384, V=32000, D=4096, dtype="bf16",
             transw="T", ignored=0.1, pad=0),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _size(rng, low, high):
    """Log-uniform; half of the sizes multiples of 64, a third of 8, a sixth any."""
    v = _log(rng, low, high)
    step = rng.choice((64, 64, 64, 8, 8, 1))
    return max(low, min(high, (v + step // 2) // step * step))


def draw(rng):
    op = rng.choice(("checkpoint", "linear8", "backward8", "loss", "loss_grad"))
    c = dict(op=op, dtype=rng.choice(("bf16", "f16")), pad=rng.choice((0, 0, 0, 8, 8, 5)))
    if op == "checkpoint":
        return c | dict(M=_log(rng, 1, 16384), N=_size(rng, 1, 14336))
    c["transw"] = rng.choice(("T", "T", "N"))
    while True:
        if op in ("linear8", "backward8"):
            c.update(M=_log(rng, 1 if op == "linear8" else 64, 16384), N=_size(rng, 64, 14336),
                     K=_size(rng, 64, 14336), act=rng.choice(ACTS))
            if op == "linear8":
                c.update(bias=rng.random() < 0.7, residual=rng.random() < 0.5)
            if c["M"] * c["N"] * c["K"] <= 16384 * 14336 * 4096:
                return c
        else:
            c.update(T=_log(rng, 1, 16384), V=_size(rng, 16, 131072), D=_size(rng, 64, 8192),
                     ignored=rng.choice((0.0, 0.1, 0.5, 0.9)))
            if c["T"] * c["V"] <= 16384 * 32000 and c["V"] * c["D"] <= 65536 * 4096 \
                    and c["T"] * c["V"] * c["D"] <= 16384 * 32000 * 4096:
                return c


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, shape, dtype, scale=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, scale, generator=g)


def _matrix(g, rows, cols, dtype, scale=1.0, pad=0):
    """rows x cols in rows of cols + pad values: a part of a wider buffer where pad > 0."""
    return _normal(g, (rows, cols + pad), dtype, scale)[:, :cols]


def _activations(g, rows, cols, dtype, pad):
    """What layers hand on: normal values, some channels twenty times as large as the others."""
    large = 1 + 19 * (torch.rand(cols + pad, generator=g, device="cuda") < 0.01)
    return _normal(g, (rows, cols + pad), dtype).mul_(large.to(dtype))[:, :cols]


def _saved(x):
    """An 8-bit checkpoint of x as a program holds it: codes in rows of whole 16 bytes, scales."""
    codes, scale = _quantise(x)
    rows = torch.zeros(x.shape[0], (x.shape[1] + 15) // 16 * 16, dtype=torch.int8, device=x.device)
    rows[:, :x.shape[1]] = codes
    return rows[:, :x.shape[1]], scale


def prepare(case, seed):
    g = _gen(seed)
    dt, pad, op = DTYPES[case["dtype"]], case["pad"], case["op"]
    if op == "checkpoint":
        return dict(case=case, x=_activations(g, case["M"], case["N"], dt, pad))
    if op in ("linear8", "backward8"):
        M, N, K = case["M"], case["N"], case["K"]
        s = dict(case=case, x=_activations(g, M, K, dt, pad))
        s["w"] = _matrix(g, *((N, K) if case["transw"] == "T" else (K, N)), dt, 1 / math.sqrt(K))
        if op == "linear8":
            s["bias"] = _normal(g, (N,), dt, 0.5) if case["bias"] else None
            s["residual"] = _matrix(g, M, N, dt, 1.0, pad) if case["residual"] else None
        else:
            s["x"] = _saved(s["x"])
            s["pre"] = _saved(_matrix(g, M, N, dt)) if case["act"] != "none" else None
            s["dy"] = _matrix(g, M, N, dt, 0.05, pad)
        return s
    T, V, D = case["T"], case["V"], case["D"]
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    w = _normal(g, (V, D), dt, 1.28 / math.sqrt(D))
    # A trained model's tokens: from ones it cannot tell to ones it is sure of.
    sure = 7.3 * torch.rand(T, 1, generator=g, device="cuda")
    x = _matrix(g, T, D, dt, 1.0, pad)
    x += (sure * w[labels].float()).to(dt)
    labels[torch.rand(T, generator=g, device="cuda") < case["ignored"]] = -100
    s = dict(case=case, x=x, labels=labels, w=w if case["transw"] == "T" else w.t().contiguous())
    if op == "loss_grad":
        s["lse"] = torch.logsumexp(x.float() @ w.float().t(), 1)
        # The mean over the counted tokens; half is trained with the loss scaled up.
        mean = (4096.0 if case["dtype"] == "f16" else 1.0) / max(1, int((labels >= 0).sum()))
        s["dloss"] = torch.full((), mean, device="cuda").expand(T)
    return s


# ---- the plain forms -------------------------------------------------------------------------

def _quantise(x):
    """(codes, scales): each row's blocks of 64 columns, by their largest magnitude. The quotient
    127 x / a of 16-bit x and a is exact enough in 32 bits that rounding it is rounding the true
    one: it is a tie exactly, or further from one than its own rounding."""
    M, N = x.shape
    blocks = (N + BLOCK - 1) // BLOCK
    v = torch.zeros(M, blocks * BLOCK, device=x.device)
    v[:, :N] = x.float()
    v = v.view(M, blocks, BLOCK)
    a = v.abs().amax(2, keepdim=True)
    codes = torch.round(v * 127 / torch.where(a == 0, torch.ones_like(a), a)).to(torch.int8)
    return codes.view(M, blocks * BLOCK)[:, :N], a[:, :, 0] / 127


def _restore(saved, dtype):
    codes, scale = saved
    return (codes.float() * scale.repeat_interleave(BLOCK, 1)[:, :codes.shape[1]]).to(dtype)


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


def _plain_checkpoint(s):
    return (_restore(_quantise(s["x"]), s["x"].dtype),)


def _plain_linear8(s):
    case, dt = s["case"], s["x"].dtype
    w = s["w"].float()
    z = s["x"].float() @ (w.t() if case["transw"] == "T" else w)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.to(dt), _restore(_quantise(z.to(dt)), dt)


def _plain_backward8(s):
    case, dt = s["case"], s["dy"].dtype
    dz = s["dy"].float()
    if s["pre"] is not None:
        dz = _act_grad(_restore(s["pre"], dt).float(), dz, case["act"])
    w, x = s["w"].float(), _restore(s["x"], dt).float()
    if case["transw"] == "T":
        dx, dw = dz @ w, dz.t() @ x
    else:
        dx, dw = dz @ w.t(), x.t() @ dz
    return dx.to(dt), dw.to(dt), dz.sum(0)


def _vocabulary(s):
    """The head's weights V x D, and which tokens count."""
    w = s["w"].float()
    return w if s["case"]["transw"] == "T" else w.t(), s["labels"] >= 0


def _plain_loss(s):
    w, counted = _vocabulary(s)
    z = s["x"].float() @ w.t()
    m = z.amax(1)
    lse = m + torch.log(torch.exp(z - m[:, None]).sum(1))
    at = torch.gather(z, 1, torch.where(counted, s["labels"], 0)[:, None])[:, 0]
    return torch.where(counted, lse - at, torch.zeros_like(lse)), lse


def _plain_loss_grad(s):
    w, counted = _vocabulary(s)
    x, dt = s["x"].float(), s["x"].dtype
    dz = torch.exp(x @ w.t() - s["lse"][:, None])
    dz.scatter_add_(1, torch.where(counted, s["labels"], 0)[:, None],
                    torch.full_like(s["lse"], -1.0)[:, None])
    dz = torch.where(counted[:, None], dz * s["dloss"][:, None], torch.zeros_like(dz))
    dx = dz @ w
    dw = dz.t() @ x if s["case"]["transw"] == "T" else x.t() @ dz
    return dx.to(dt), dw.to(dt)


PLAIN = {"checkpoint": _plain_checkpoint, "linear8": _plain_linear8, "backward8": _plain_backward8,
         "loss": _plain_loss, "loss_grad": _plain_loss_grad}


def _own(s):
    import dense_fp32_gemm_08_gb300 as sg
    case, op = s["case"], s["case"]["op"]
    if op == "checkpoint":
        return (sg.restore8(sg.checkpoint8(s["x"])),)
    if op == "linear8":
        y, pre = sg.linear(s["x"], s["w"], bias=s["bias"], act=case["act"], residual=s["residual"],
                           transw=case["transw"], save_pre="8bit")
        return y, sg.restore8(pre)
    if op == "backward8":
        dt = s["dy"].dtype
        pre = None if s["pre"] is None else sg.Checkpoint8(*s["pre"], dt)
        return sg.linear_backward(s["dy"], sg.Checkpoint8(*s["x"], dt), s["w"], pre=pre,
                                  act=case["act"], transw=case["transw"])
    if op == "loss":
        return sg.cross_entropy(s["x"], s["w"], s["labels"], transw=case["transw"])
    return sg.cross_entropy_backward(s["dloss"], s["x"], s["w"], s["labels"], s["lse"],
                                     transw=case["transw"])


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["case"]["op"]](state)


def work(case):
    op = case["op"]
    if op in ("loss", "loss_grad"):
        T, V, D = case["T"], case["V"], case["D"]
        if op == "loss":
            return {"bytes": 2 * (T * D + V * D) + 16 * T, "flops": 2 * T * V * D}
        # The logits once more, since they are not kept, and the two products.
        return {"bytes": 4 * (T * D + V * D) + 16 * T, "flops": 6 * T * V * D}
    M, N = case["M"], case["N"]

    def saved(rows, cols):
        return rows * cols + 4 * rows * -(-cols // BLOCK)

    if op == "checkpoint":  # written when it is saved, read when it is restored
        return {"bytes": 4 * M * N + 2 * saved(M, N), "flops": 4 * M * N}
    K = case["K"]
    if op == "linear8":
        return {"bytes": 2 * (M * K + N * K + M * N * (2 + case["residual"]) + N * case["bias"])
                + 2 * saved(M, N), "flops": 2 * M * N * K}
    return {"bytes": 2 * (M * N + M * K + 2 * N * K) + saved(M, K)
            + (saved(M, N) if case["act"] != "none" else 0) + 4 * N, "flops": 4 * M * N * K}


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


def _exact_checkpoint(x):
    """What an 8-bit checkpoint of x stands for."""
    out = torch.empty_like(x)
    for c in range(0, x.shape[1], BLOCK):
        part = x[:, c:c + BLOCK]
        top = part.abs().max(dim=1, keepdim=True).values
        step = top / 127
        out[:, c:c + BLOCK] = torch.where(top > 0, torch.round(part * 127 / top) * step, 0.0)
    return out


def _exact_restore(saved):
    codes, scale = saved
    out = codes.double()
    for b in range(scale.shape[1]):
        out[:, b * BLOCK:(b + 1) * BLOCK] *= scale[:, b:b + 1].double()
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]

    def wide(t):
        return t.double()

    if op == "checkpoint":
        return (_exact_checkpoint(wide(s["x"])),)
    w = wide(s["w"]) if case["transw"] == "N" else wide(s["w"]).T
    if op == "linear8":
        z = torch.mm(wide(s["x"]), w)
        if s["bias"] is not None:
            z += wide(s["bias"])
        y = _exact_act(z, case["act"])
        if s["residual"] is not None:
            y = y + wide(s["residual"])
        # The checkpoint is of the pre-activation in 16 bits, as the layer would keep it.
        return y, _exact_checkpoint(wide(z.to(s["x"].dtype)))
    if op == "backward8":
        dy = wide(s["dy"])
        if s["pre"] is not None:  # the slope by torch's own differentiation, in 64 bits
            z = _exact_restore(s["pre"]).to(s["dy"].dtype).double().requires_grad_()
            if case["act"] == "relu":
                dy = dy * (z.detach() > 0)
            else:
                dy, = torch.autograd.grad(_exact_act(z, case["act"]), z, dy)
        dx = torch.mm(dy, w.T)
        dw = torch.mm(_exact_restore(s["x"]).T, dy)
        return dx, dw if case["transw"] == "N" else dw.T.contiguous(), dy.sum(dim=0)
    x, labels = wide(s["x"]), s["labels"]
    rows = torch.nonzero(labels >= 0)[:, 0]
    if op == "loss":
        logp = torch.mm(x, w)
        lse = torch.logsumexp(logp, dim=1)
        loss = torch.zeros_like(lse)
        loss[rows] = lse[rows] - logp[rows, labels[rows]]
        return loss, lse
    share = torch.exp(torch.mm(x[rows], w) - wide(s["lse"])[rows, None])
    share[torch.arange(len(rows), device=x.device), labels[rows]] -= 1
    share *= wide(s["dloss"])[rows, None]
    dx = torch.zeros_like(x)
    dx[rows] = torch.mm(share, w.T)
    dw = torch.mm(x[rows].T, share)
    return dx, dw if case["transw"] == "N" else dw.T.contiguous()
