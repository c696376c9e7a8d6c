"""Plain 64-bit definitions of the layer operators on 16-bit values, and the tolerances their
results are held to.

Tolerances, derived before any run. u is the unit roundoff of the type (2^-8 for bfloat16,
2^-11 for half) and tiny half its smallest subnormal step. An output is rounded once: u |ref|.
A product's fp32 sum is held to the bound of the library's fp32 products, ACC = 1e-5 times the
sum of absolute products (plus |bias|); an activation passes an input error on scaled by at most
1.2 and adds a few fp32 ulps of (1 + |z|). Where an intermediate matrix is handed to the tensor
cores in 16 bits (dz of the gradient, h of the mixture of experts), each of its values is off by
u |value| + tiny, and the product passes that on through the absolute values of its other
factor."""
from __future__ import annotations

import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}
ACC = 1e-5
ULPS = 16 * 2.0 ** -24


def act(z, name):
    if name == "relu":
        return torch.where(z <= 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if name == "silu":
        return z / (1 + torch.exp(-z))
    return z


def act_grad(z, name):
    """act'(z), from the formulas."""
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    return torch.ones_like(z)


def weight_nk(w, transw):
    """op(W)^T, N x K."""
    return w.double() if transw == "T" else w.double().t()


def linear_ref(x, w, bias, name, res, transw):
    """(y, z) in 64 bits and the tolerances of each."""
    xd, wd, dt = x.double(), weight_nk(w, transw), x.dtype
    z = xd @ wd.t()
    zerr = ACC * (xd.abs() @ wd.abs().t())
    if bias is not None:
        z = z + bias.double()
        zerr = zerr + ACC * bias.double().abs()
    y = act(z, name)
    yerr = zerr * (1.0 if name == "none" else 1.2)
    if name != "none":
        yerr = yerr + ULPS * (1 + z.abs())
    if res is not None:
        y = y + res.double()
        yerr = yerr + 2.0 ** -23 * y.abs()
    u, tiny = U[dt] * 1.001, TINY[dt]
    return y, z, yerr + u * y.abs() + tiny, zerr + u * z.abs() + tiny


def backward_ref(dy, x, w, pre, name, transw):
    """(dx, dw, db) in 64 bits and their tolerances."""
    dt = x.dtype
    u, tiny = U[dt] * 1.001, TINY[dt]
    xd, wd, dz = x.double(), weight_nk(w, transw), dy.double()
    derr = torch.zeros_like(dz)
    serr = derr
    if name != "none":
        z = pre.double()
        serr = ULPS * dz.abs() * (1 + z.abs())
        dz = dz * act_grad(z, name)
        derr = serr + u * dz.abs() + tiny
    dx = dz @ wd
    dxerr = derr @ wd.abs() + ACC * (dz.abs() @ wd.abs()) + u * dx.abs() + tiny
    dw = dz.t() @ xd
    dwerr = derr.t() @ xd.abs() + ACC * (dz.abs().t() @ xd.abs()) + u * dw.abs() + tiny
    if transw == "N":
        dw, dwerr = dw.t(), dwerr.t()
    return dx, dw, dz.sum(0), dxerr, dwerr, serr.sum(0) + ACC * dz.abs().sum(0) + 1e-30


def moe_ref(x, router, w_gate, w_up, w_down, topk, name, renormalize, active, res):
    """(y, index, weight) in 64 bits and the tolerances of y and weight."""
    dt = x.dtype
    u, tiny = U[dt] * 1.001, TINY[dt]
    T, E, xd = x.shape[0], router.shape[0], x.double()
    score = xd @ router.double().t()
    serr = ACC * (xd.abs() @ router.double().abs().t())
    index = torch.full((T, topk), -1, dtype=torch.int32, device=x.device)
    weight = torch.zeros((T, topk), dtype=torch.float64, device=x.device)
    werr = torch.zeros_like(weight)
    y = torch.zeros_like(xd) if res is None else res.double().clone()
    yerr = 2.0 ** -22 * y.abs()
    for t in range(T):
        if active is not None and not bool(active[t]):
            continue
        row = score[t].tolist()
        best = sorted(range(E), key=lambda e: (-row[e], e))[:topk]
        p = torch.softmax(score[t], 0)[best]
        w = p / p.sum() if renormalize else p
        index[t] = torch.tensor(best, dtype=torch.int32)
        weight[t] = w
        # p's relative error: twice the scores' error (its own and the largest term's), plus ulps
        werr[t] = w * (4 * float(serr[t].max()) + ULPS)
        for j, e in enumerate(best):
            up = w_up[e].double()
            v = up @ xd[t]
            verr = ACC * (up.abs() @ xd[t].abs())
            if w_gate is not None:
                gt = w_gate[e].double()
                g = gt @ xd[t]
                gerr = ACC * (gt.abs() @ xd[t].abs())
                a = act(g, name)
                h = a * v
                herr = a.abs() * verr + (1.2 * gerr + ULPS * (1 + g.abs())) * (v.abs() + verr)
            else:
                h = act(v, name)
                herr = 1.2 * verr + ULPS * (1 + v.abs())
            herr = herr + u * h.abs() + tiny
            dn = w_down[e].double()
            o = dn @ h
            oerr = dn.abs() @ herr + ACC * (dn.abs() @ h.abs())
            y[t] += w[j] * o
            yerr[t] += w[j] * oerr + werr[t, j] * o.abs()
    return y, index, weight, yerr + u * y.abs() + tiny, werr


def worst(got, ref, tol):
    """Largest error as a multiple of its tolerance (infinite where NaN or Inf do not agree)."""
    got = got.double()
    fine = torch.isfinite(ref)
    if got.shape != ref.shape or not torch.equal(fine, torch.isfinite(got)):
        return math.inf
    if not bool(fine.any()):
        return 0.0
    return float(((got - ref).abs() / tol)[fine].max())
