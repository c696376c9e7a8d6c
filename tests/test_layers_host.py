"""Refusals and degenerate calls of the layer operators, without a GPU."""
from __future__ import annotations

import pytest

FAKE = 1 << 20  # a 16-byte aligned non-null address; argument checks never dereference it

LINEAR = ["dtype", "transw", "M", "N", "K", "X", "ldx", "W", "ldw", "bias", "act", "R", "ldr", "Y", "ldy", "Z",
          "ldz", "stream"]
LINEAR_OK = dict(dtype=0, transw=1, M=8, N=6, K=4, X=FAKE, ldx=4, W=FAKE, ldw=4, bias=None, act=0, R=None, ldr=0,
                 Y=FAKE, ldy=6, Z=None, ldz=0, stream=None)
BACKWARD = ["dtype", "transw", "M", "N", "K", "dY", "lddy", "Z", "ldz", "act", "X", "ldx", "W", "ldw", "dX", "lddx",
            "dW", "lddw", "db", "stream"]
BACKWARD_OK = dict(dtype=1, transw=1, M=8, N=6, K=4, dY=FAKE, lddy=6, Z=FAKE, ldz=6, act=2, X=FAKE, ldx=4, W=FAKE,
                   ldw=4, dX=FAKE, lddx=4, dW=FAKE, lddw=4, db=FAKE, stream=None)
MOE = ["dtype", "act", "T", "E", "topk", "D", "F", "X", "ldx", "Wr", "ldwr", "Wgate", "Wup", "ldu", "strideu", "Wdown",
       "ldd", "strided", "renormalize", "active", "R", "ldr", "Y", "ldy", "topk_index", "topk_weight", "stream"]
MOE_OK = dict(dtype=0, act=4, T=3, E=4, topk=2, D=16, F=24, X=FAKE, ldx=16, Wr=FAKE, ldwr=16, Wgate=FAKE, Wup=FAKE,
              ldu=16, strideu=384, Wdown=FAKE, ldd=24, strided=384, renormalize=1, active=None, R=None, ldr=0, Y=FAKE,
              ldy=16, topk_index=None, topk_weight=None, stream=None)


def call(sg, name, order, base, **change):
    args = dict(base, **change)
    return getattr(sg.lib(), name)(*(args[n] for n in order))


def refused(sg, name, order, base, why, status=1, **change):
    assert call(sg, name, order, base, **change) == status, change
    assert why in sg.sgemm_last_error(), (change, sg.sgemm_last_error())


@pytest.mark.parametrize("change,why", [
    (dict(dtype=2), "dtype"), (dict(dtype=-1), "dtype"), (dict(transw=2), "transw"), (dict(act=5), "activation"),
    (dict(act=-1), "activation"), (dict(M=-1), "M, N and K"), (dict(K=-1), "M, N and K"), (dict(ldx=3), "ldx"),
    (dict(ldw=3), "ldw"), (dict(transw=0, ldw=5), "ldw"), (dict(R=FAKE, ldr=5), "ldr"), (dict(ldy=5), "ldy"),
    (dict(Z=FAKE + 64, ldz=5), "ldz"), (dict(Y=None), "Y is NULL"), (dict(X=None), "X or W"), (dict(W=None), "X or W"),
    (dict(X=FAKE + 1), "aligned"), (dict(bias=FAKE + 3), "aligned"), (dict(Z=FAKE, ldz=6), "same matrix"),
    (dict(R=FAKE, ldr=8), "overlaps"), (dict(K=0, ldx=0), "ldx"),
])
def test_linear_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_linear", LINEAR, LINEAR_OK, why, **change)


@pytest.mark.parametrize("change,why", [
    (dict(dtype=7), "dtype"), (dict(transw=-1), "transw"), (dict(act=9), "activation"), (dict(N=-2), "M, N and K"),
    (dict(lddy=5), "lddy"), (dict(ldz=5), "ldz"), (dict(ldx=3), "ldx"), (dict(ldw=3), "ldw"), (dict(lddx=3), "lddx"),
    (dict(lddw=3), "lddw"), (dict(transw=0, ldw=6, lddw=5), "lddw"), (dict(dY=None), "dY is NULL"),
    (dict(Z=None), "Z is NULL"), (dict(X=None), "X is NULL"), (dict(W=None), "W is NULL"), (dict(dX=FAKE + 1), "aligned"),
    (dict(db=FAKE + 2), "aligned"),
])
def test_backward_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_linear_backward", BACKWARD, BACKWARD_OK, why, **change)


@pytest.mark.parametrize("change,why", [
    (dict(dtype=2), "dtype"), (dict(act=5), "activation"), (dict(T=-1), "T, D and F"), (dict(F=-1), "T, D and F"),
    (dict(E=0), "E must"), (dict(topk=0), "topk"), (dict(topk=5), "topk"), (dict(ldx=15), "ldx"),
    (dict(ldwr=15), "ldwr"), (dict(ldu=15), "ldu"), (dict(ldd=23), "ldd"), (dict(strideu=383), "strideu"),
    (dict(strided=383), "strided"), (dict(R=FAKE, ldr=15), "ldr"), (dict(ldy=15), "ldy"), (dict(Y=None), "Y is NULL"),
    (dict(X=None), "X or Wr"), (dict(Wr=None), "X or Wr"), (dict(Wup=None), "Wup or Wdown"),
    (dict(Wdown=None), "Wup or Wdown"), (dict(Wgate=FAKE + 1), "aligned"), (dict(topk_index=FAKE + 2), "aligned"),
    (dict(R=FAKE, ldr=24), "overlaps"),
])
def test_moe_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_moe", MOE, MOE_OK, why, **change)


@pytest.mark.parametrize("change", [dict(T=65), dict(E=513), dict(E=32, topk=17)])
def test_moe_limits(sgemm_lib, change):
    refused(sgemm_lib, "sgemm_moe", MOE, MOE_OK, "at most", status=4, **change)


def test_oversized_dimension_is_unsupported(sgemm_lib):
    refused(sgemm_lib, "sgemm_linear", LINEAR, LINEAR_OK, "2^31", status=4, M=1 << 31)
    refused(sgemm_lib, "sgemm_linear_backward", BACKWARD, BACKWARD_OK, "2^31", status=4, M=1 << 31)


def test_degenerate_calls_need_no_device(sgemm_lib):
    for change in (dict(M=0), dict(N=0, ldy=1, transw=0, ldw=1)):
        assert call(sgemm_lib, "sgemm_linear", LINEAR, LINEAR_OK, X=None, W=None, Y=None, **change) == 0
    nothing = dict(dX=None, dW=None, db=None)
    assert call(sgemm_lib, "sgemm_linear_backward", BACKWARD, BACKWARD_OK, **nothing) == 0
    assert call(sgemm_lib, "sgemm_linear_backward", BACKWARD, BACKWARD_OK, M=0, dW=None, db=None) == 0
    assert call(sgemm_lib, "sgemm_moe", MOE, MOE_OK, T=0, X=None, Y=None) == 0


def test_python_shapes_and_types(sgemm_lib):
    torch = pytest.importorskip("torch")
    sg = sgemm_lib
    x, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    with pytest.raises(TypeError):  # host tensors
        sg.linear(x, w)
    for bad in (dict(weight=w[:, :7]), dict(weight=w, bias=x[0]), dict(weight=w, residual=x),
                dict(weight=w.t(), transw="T"), dict(weight=w, out=x)):
        with pytest.raises(ValueError):
            sg.linear(x, **bad)
    with pytest.raises(ValueError):  # rows not contiguous
        sg.linear(torch.zeros(8, 3, dtype=torch.bfloat16).t(), w)
    with pytest.raises(ValueError):
        sg.linear_backward(x, x, w)
    with pytest.raises(ValueError):
        sg.moe(x, w, None, torch.zeros(4, 6, 8), torch.zeros(4, 8, 6), 1)
