"""The layer operators' activations over their whole range, tails included, against 64 bits.

Tolerances, derived before any run. An activation is evaluated in fp32 to REL |act(z)|: a fit of
5.9e-6, the rounded argument of an exponential (z^2 / 2 <= 72 at |z| = 12, two roundings of 2^-24: 9e-6;
2u <= 88 for the tanh form while its value is representable, seven roundings: 3.7e-5) and a few ulps.
Results below the smallest normal fp32 number are 0, times |z| <= 12 and, for a slope, a
factor of 400 at most (z (2u)' of the tanh form). The result is then rounded once: u |act(z)|, or half
the smallest subnormal step. A slope is the sum of two terms, each to REL of itself; and, as its sums
leave in 32 bits, to 16 fp32 ulps of 1 and of what an ulp of the sigmoid or of Phi is multiplied by (|z| times
the slope of its argument)."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import layer_case as ref  # noqa: E402

pytestmark = pytest.mark.gpu

REL = 4e-5
FLUSH = 2.0 ** -126
DTYPES = [torch.bfloat16, torch.float16]
ACTS = ["relu", "gelu", "gelu_tanh", "silu"]


def sweep(dtype):
    """Every value of the type in [-12, 12] that a step of 2^-9 meets, and small ones."""
    z = torch.arange(-12 * 512, 12 * 512 + 1, device="cuda").double() / 512
    small = 2.0 ** -torch.arange(0, 24, device="cuda").double()
    return torch.unique(torch.cat([z, small, -small]).to(dtype).double()).to(dtype)


def act(z, name):
    """act(z) in 64 bits without cancellation in the tails."""
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * torch.sigmoid(z)
    return torch.where(z <= 0, torch.zeros_like(z), z)


def slope(z, name):
    """act'(z), the sum of its two terms' absolute values, and the factor of an ulp's error in it."""
    factor = z.abs()
    if name == "gelu":
        a, b = 0.5 * torch.special.erfc(-z / math.sqrt(2.0)), z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    elif name == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        a = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        b = z * a * torch.sigmoid(-c * (z + 0.044715 * z ** 3)) * c * (1 + 3 * 0.044715 * z * z)
        factor = z.abs() * c * (1 + 3 * 0.044715 * z * z)
    elif name == "silu":
        a, b = torch.sigmoid(z), z * torch.sigmoid(z) * torch.sigmoid(-z)
    else:
        a, b = (z > 0).double(), torch.zeros_like(z)
    return a + b, a.abs() + b.abs(), 1 + factor


def check(got, z, name, dtype):
    want = act(z.double(), name)
    tol = (REL + ref.U[dtype] * 1.001) * want.abs() + ref.TINY[dtype] + 12 * FLUSH
    assert ref.worst(got, want, tol) <= 1.0, (ref.worst(got, want, tol), name)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("M,K", [(1, 0), (3, 8), (40, 16), (300, 8)])
def test_activations_to_their_rounding(sgemm_lib, dtype, name, M, K):
    """z as the bias of a product of zeros: no product, few rows, more rows, pairs of CTAs."""
    z = sweep(dtype)
    x = torch.zeros(M, K, dtype=dtype, device="cuda")
    w = torch.ones(z.numel(), K, dtype=dtype, device="cuda")
    got = sgemm_lib.linear(x, w, bias=z, act=name)
    for row in (0, M - 1):
        check(got[row], z, name, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("width", [264, 263])
def test_activations_of_experts(sgemm_lib, dtype, name, width):
    """One expert whose first matrix has z in its first column and whose second is the unit matrix,
    in rows that TMA can address and in rows that it cannot."""
    zs = sweep(dtype)
    for z in zs[::5].split(width):
        n = z.numel()
        x = torch.zeros(1, width, dtype=dtype, device="cuda")
        x[0, 0] = 1
        up = torch.zeros(1, width, width, dtype=dtype, device="cuda")
        up[0, :n, 0] = z
        down = torch.eye(width, dtype=dtype, device="cuda")[None]
        y, _, _ = sgemm_lib.moe(x, torch.zeros_like(x), None, up, down, 1, act=name)
        check(y[0, :n], z, name, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("name", ACTS)
def test_slopes(sgemm_lib, dtype, name):
    """The bias' gradient of one row of ones is act'(z) in 32 bits."""
    z = sweep(dtype)
    n = z.numel()
    for part in (z, z[: n // 8 * 8]):  # rows of 2-byte and of 16-byte loads
        dy = torch.ones(1, part.numel(), dtype=dtype, device="cuda")
        x, w = torch.ones(1, 8, dtype=dtype, device="cuda"), torch.ones(part.numel(), 8, dtype=dtype, device="cuda")
        _, _, db = sgemm_lib.linear_backward(dy, x, w, pre=part[None].contiguous(), act=name, need_dx=False,
                                             need_dw=False)
        want, size, factor = slope(part.double(), name)
        tol = torch.minimum(REL * size + 2.0 ** -23 * want.abs(), ref.ULPS * factor) + 400 * FLUSH
        assert ref.worst(db, want, tol) <= 1.0, (ref.worst(db, want, tol), name)
