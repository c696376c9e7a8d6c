"""GPU parity of the head's cross entropy where its values are not finite or its labels all but certain."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16]
# Few tokens, more of them on the streaming product, and the pair product (more than 128 tiles of 64 x 128).
TOKENS_AND_ENTRIES = [(3, 300), (140, 700), (700, 3001)]


def normal(seed, *shape, dtype=torch.bfloat16, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def inputs(T, V, D, dtype=torch.bfloat16, transw="T", seed=0):
    x = normal(seed + 1, T, D, dtype=dtype)
    w = normal(seed + 2, V, D, dtype=dtype, scale=1.5 / math.sqrt(D))
    g = torch.Generator(device="cuda").manual_seed(seed)
    labels = torch.randint(V, (T,), generator=g, device="cuda")
    return x, w if transw == "T" else w.t().contiguous(), labels


@pytest.mark.parametrize("T,V", TOKENS_AND_ENTRIES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_a_token_with_a_nan_has_nan_lse(sgemm_lib, dtype, T, V):
    """Every logit of the token is NaN: lse too, whether or not the token counts, and no other token's."""
    sg = sgemm_lib
    x, w, labels = inputs(T, V, 72, dtype, seed=T)
    want_loss, want_lse = sg.cross_entropy(x, w, labels)
    x[0, 3], x[2, 70] = math.nan, math.nan
    labels[2] = -100
    loss, lse = sg.cross_entropy(x, w, labels)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
    assert bool(torch.isnan(lse[0])) and bool(torch.isnan(lse[2]))
    assert bool(torch.isnan(loss[0])) and float(loss[2]) == 0.0
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[0] = keep[2] = False
    assert torch.equal(lse[keep], want_lse[keep]) and torch.equal(loss[keep], want_loss[keep])
    alone = torch.empty_like(lse)
    sg.sgemm_cross_entropy("bf16" if dtype is torch.bfloat16 else "f16", "T", T, V, 72, x, 72, w, 72, labels, None, alone)
    assert torch.equal(alone.isnan(), lse.isnan()) and torch.equal(alone[keep], lse[keep])
