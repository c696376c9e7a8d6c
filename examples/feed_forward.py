"""A model's feed-forward half on this library's layer operators: a dense block trained for a few
steps with sgemm_linear and its gradients, then a block of experts serving single tokens.

    python examples/feed_forward.py            # needs a GB300 and the built library
"""
from __future__ import annotations

import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import dense_fp32_gemm_08_gb300 as sg  # noqa: E402


class Linear(torch.autograd.Function):
    """act(x W^T + b) + residual; the weight is stored out x in, as torch.nn.Linear keeps it."""

    @staticmethod
    def forward(ctx, x, weight, bias, act, residual):
        keep = act != "none"
        out = sg.linear(x, weight, bias=bias, act=act, residual=residual, save_pre=keep)
        y, pre = out if keep else (out, None)
        ctx.save_for_backward(x, weight, pre)
        ctx.act = act
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, pre = ctx.saved_tensors
        need_x, need_w, need_b, _, need_r = ctx.needs_input_grad
        dy = dy.contiguous()
        dx, dw, db = sg.linear_backward(dy, x, weight, pre=pre, act=ctx.act, need_dx=need_x,
                                        need_dw=need_w, need_db=need_b)
        return dx, dw, None if db is None else db.to(dy.dtype), None, dy if need_r else None


def block(x, p):
    """x + W2 gelu(W1 x + b1) + b2"""
    h = Linear.apply(x, p["w1"], p["b1"], "gelu", None)
    return Linear.apply(h, p["w2"], p["b2"], "none", x)


def train(steps=12, rows=512, width=512, hidden=2048, rate=2.0, seed=0):
    """Fits the block to a fixed random target; returns the losses."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).bfloat16()

    # 32-bit master weights; the layers see them in 16 bits.
    master = {"w1": normal(hidden, width, scale=width ** -0.5), "b1": normal(hidden, scale=0.1),
              "w2": normal(width, hidden, scale=hidden ** -0.5), "b2": normal(width, scale=0.1)}
    master = {name: v.float() for name, v in master.items()}
    x, target = normal(rows, width), normal(rows, width)
    losses = []
    for _ in range(steps):
        p = {name: v.bfloat16().requires_grad_() for name, v in master.items()}
        loss = (block(x, p).float() - target.float()).square().mean()
        grads = torch.autograd.grad(loss, list(p.values()))
        for v, d in zip(master.values(), grads):
            v -= rate * d.float()
        losses.append(float(loss.detach()))
    return losses


def serve(tokens=4, width=1024, hidden=2816, experts=16, topk=2, seed=1):
    """One decoding step of a few tokens: a projection, then the experts with the projection's output
    as their residual. Returns the step's output and the experts that each token chose."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale=1.0):
        return torch.empty(*shape, dtype=torch.bfloat16, device="cuda").normal_(0.0, scale, generator=g)

    x = normal(tokens, width)
    w_out = normal(width, width, scale=width ** -0.5)
    router = normal(experts, width, scale=width ** -0.5)
    gate, up = (normal(experts, hidden, width, scale=width ** -0.5) for _ in range(2))
    down = normal(experts, width, hidden, scale=hidden ** -0.5)
    h = sg.linear(x, w_out, residual=x)
    y, index, weight = sg.moe(h, router, gate, up, down, topk, act="silu", residual=h)
    return y, index, weight


def main():
    losses = train()
    print("training loss:", " ".join(f"{v:.4f}" for v in losses))
    y, index, weight = serve()
    print("experts per token:", index.tolist())
    print("their weights:", [[round(w, 3) for w in row] for row in weight.tolist()])
    print("output norm per token:", [round(v, 2) for v in y.float().norm(dim=1).tolist()])
    status = sg.sgemm_device_status()
    if status != sg.SGEMM_OK:
        raise RuntimeError(f"device status {status}")


if __name__ == "__main__":
    main()
