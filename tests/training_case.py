"""Plain 64-bit definitions of the 8-bit checkpoints and of the head's cross entropy, and the tolerances
their results are held to.

A checkpoint is held to its definition exactly: its quotient is rounded as the true one is. (127 x / a of
16-bit x and a: in 64 bits the quotient of two integers below 2^18 and 2^11, shifted, is nearer to a tie
than its rounding error only when it is one.)

The loss, derived before any run. A logit's fp32 product is held to ACC times the sum of absolute
products, as the library's other products. With e that bound, a term exp(z - m) is off by a factor
exp(e), 2^-22 of the hardware's exponential and |z - m| 2^-22 of its argument's rounding, and the sums
add positive terms: 64 of a warp's columns one after the other, then parts of 64 columns, a 32nd of
them one after the other (each join an exponential and two roundings). An argument of size a counts with
weight exp(-a), so a exp(-a) < 0.4 bounds its share. So
    |lse's error| <= max e + (64 + parts / 32 * 8 + 16) 2^-24 + 2^-22 |lse|,
and the loss adds its label's e and a rounding of |lse| + |z|.

The gradient. p = exp(z - lse) is off by p (e + 2^-22 + |z - lse| 2^-22 + 2^-23 (|z| + |lse|)) (the last: the
subtraction's operands are fp32), 1 is subtracted exactly to 2^-24 (or expm1 taken, which is nearer), and dz is rounded to 16 bits: u |dz|,
and in half half a subnormal step over the factor that brings the largest |dloss| to 2^14. The products
pass that on through the absolute values of their other factor, with ACC and one rounding of their own."""
from __future__ import annotations

import torch

from layer_case import ACC, TINY, U, weight_nk


def checkpoint_ref(x):
    """(codes, scale, restored): int8, float32 and x's type."""
    M, N = x.shape
    blocks = -(-N // 64)
    codes = torch.zeros(M, N, dtype=torch.int8, device=x.device)
    scale = torch.zeros(M, blocks, dtype=torch.float32, device=x.device)
    restored = torch.zeros_like(x)
    for b in range(blocks):
        part = x[:, 64 * b:64 * b + 64].double()
        top = part.abs().amax(1, keepdim=True)  # NaN stays
        fine = torch.isfinite(top)
        safe = torch.where(fine & (top > 0), top, 1.0)
        q = torch.where(fine & (top > 0), torch.round(127 * part / safe), 0.0)
        s = torch.where(fine, top / 127, float("nan")).float()
        codes[:, 64 * b:64 * b + 64] = q.to(torch.int8)
        scale[:, b] = s[:, 0]
        restored[:, 64 * b:64 * b + 64] = (q.float() * s).to(x.dtype)
    return codes, scale, restored


def head_ref(x, w, labels, transw):
    """(loss, lse, z) in 64 bits, and the tolerances of loss, lse and z."""
    xd, wd = x.double(), weight_nk(w, transw)
    V = wd.shape[0]
    z = xd @ wd.t()
    e = ACC * (xd.abs() @ wd.abs().t())
    lse = torch.logsumexp(z, 1)
    parts = -(-V // 64)
    ltol = e.amax(1) + (64 + parts / 32 * 8 + 16) * 2.0 ** -24 + 2.0 ** -22 * lse.abs()
    counts = (labels >= 0) & (labels < V)
    at = torch.where(counts, labels, 0)[:, None]
    zl = z.gather(1, at)[:, 0]
    loss = torch.where(counts, lse - zl, 0.0)
    tol = torch.where(counts, ltol + e.gather(1, at)[:, 0] + 2.0 ** -23 * (lse.abs() + zl.abs()), 1e-300)
    return loss, lse, z, tol, ltol, e


def head_grad_ref(dloss, x, w, labels, lse, transw):
    """(dx, dw) in 64 bits from the fp32 lse, and their tolerances."""
    dt = x.dtype
    u, tiny = U[dt] * 1.001, TINY[dt]
    xd, wd, ld, dl = x.double(), weight_nk(w, transw), lse.double()[:, None], dloss.double()[:, None]
    V = wd.shape[0]
    z = xd @ wd.t()
    e = ACC * (xd.abs() @ wd.abs().t())
    counts = ((labels >= 0) & (labels < V))[:, None]
    p = torch.exp(z - ld)
    perr = p * (e + 2.0 ** -22 * (1 + (z - ld).abs()) + 2.0 ** -23 * (z.abs() + ld.abs()))
    hot = torch.zeros_like(p).scatter_(1, torch.where(counts, labels[:, None], 0), 1.0)
    dz = torch.where(counts, dl * (p - hot), 0.0)
    largest = float((dl.abs() * counts).amax()) if dl.numel() else 0.0
    step = tiny if dt == torch.bfloat16 else 2.0 ** -25 * largest * 2.0 ** -14 * 1.01 + 1e-45
    derr = torch.where(counts, dl.abs() * (perr + 2.0 ** -24 * hot) + 2.0 ** -22 * dz.abs(), 0.0)
    derr = torch.where(counts, derr + u * dz.abs() + step, 0.0)
    dx = dz @ wd
    dxerr = derr @ wd.abs() + ACC * (dz.abs() @ wd.abs()) + u * dx.abs() + tiny
    dw = dz.t() @ xd
    dwerr = derr.t() @ xd.abs() + ACC * (dz.abs().t() @ xd.abs()) + u * dw.abs() + tiny
    if transw == "N":
        dw, dwerr = dw.t(), dwerr.t()
    return dx, dw, dxerr, dwerr
