"""Experts in half whose hidden values exceed the type's range (65,504) while the outputs do not."""
from __future__ import annotations

import math

import pytest

torch = pytest.importorskip("torch")

import layer_case as ref  # noqa: E402

pytestmark = pytest.mark.gpu


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).half()


def shifted(t, pad):
    """The same values in rows that TMA can (pad 0) or cannot address."""
    if pad == 0:
        return t
    wide = torch.zeros(*t.shape[:-1], t.shape[-1] + pad, dtype=t.dtype, device="cuda")
    wide[..., : t.shape[-1]] = t
    return wide[..., : t.shape[-1]]


def layer(seed, T, E, D, F, gated, large, down):
    """Every second token is `large` times as long as the others."""
    x = normal(seed, T, D)
    big = x.clone()
    big[::2] *= large
    router = normal(seed + 1, E, D, scale=0.5 / math.sqrt(D) / large)
    gate = normal(seed + 2, E, F, D, scale=10 / math.sqrt(D)) if gated else None
    return x, big, router, gate, normal(seed + 3, E, F, D, scale=10 / math.sqrt(D)), normal(seed + 4, E, D, F, scale=down)


SIZES = [(1, 4, 2, 128, 264), (3, 4, 2, 128, 264), (24, 16, 4, 264, 200), (64, 8, 4, 136, 520), (2, 2, 1, 64, 20040),
         (17, 60, 6, 512, 128), (40, 4, 2, 1024, 1024)]


@pytest.mark.parametrize("T,E,k,D,F", SIZES)
@pytest.mark.parametrize("gated,act,large,down", [(True, "silu", 30.0, 1e-3), (True, "gelu", 1000.0, 1e-6),
                                                  (False, "none", 1e4, 1e-3)])
@pytest.mark.parametrize("pad", [0, 3])
def test_hidden_values_past_the_range_of_half(sgemm_lib, T, E, k, D, F, gated, act, large, down, pad):
    sg = sgemm_lib
    x, big, router, gate, up, dn = layer(7, T, E, D, F, gated, large, down)
    weights = [None if w is None else shifted(w, pad) for w in (gate, up, dn)]
    u = big.double() @ up.double().transpose(1, 2)
    h = u if gate is None else ref.act(big.double() @ gate.double().transpose(1, 2), act) * u
    assert float(h.abs().max()) > 65504
    before = sg.moe(x, router, *weights, k, act=act)
    for _ in range(2):
        got = sg.moe(big, router, *weights, k, act=act, residual=x)
        assert sg.sgemm_device_status() == sg.SGEMM_OK
        y, index, weight, ytol, wtol = ref.moe_ref(big, router, gate, up, dn, k, act, True, None, x)
        assert bool(torch.isfinite(y).all()) and float(y.abs().max()) < 65504
        assert torch.equal(got[1], index) and ref.worst(got[2], weight, wtol + 1e-12) <= 1.0
        assert ref.worst(got[0], y, ytol) <= 1.0, ref.worst(got[0], y, ytol)
    again = sg.moe(x, router, *weights, k, act=act)  # nothing is left behind
    assert all(torch.equal(a, b) for a, b in zip(before, again))


def test_infinite_rows_stay_infinite_and_apart(sgemm_lib):
    sg = sgemm_lib
    T, E, D, F = 6, 4, 128, 264
    x, big, router, gate, up, down = layer(3, T, E, D, F, True, 30.0, 1e-3)
    active = torch.ones(T, dtype=torch.bool, device="cuda")
    active[5] = False
    clean = sg.moe(big, router, gate, up, down, 2, active=active)
    big[1, 3] = math.inf
    big[5] = math.nan
    got = sg.moe(big, router, gate, up, down, 2, active=active)
    keep = [0, 2, 3, 4]
    assert bool(torch.isfinite(clean[0]).all())
    assert not bool(torch.isfinite(got[0][1]).any()) and not bool(got[0][5].any())
    assert torch.allclose(got[0][keep].float(), clean[0][keep].float(), rtol=2.0 ** -9, atol=1e-2)
    assert sg.sgemm_device_status() == sg.SGEMM_OK
