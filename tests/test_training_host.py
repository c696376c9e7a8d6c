"""Refusals and degenerate calls of the 8-bit checkpoints and of the head's cross entropy, without a GPU."""
from __future__ import annotations

import pytest

from test_layers_host import FAKE, BACKWARD_OK, LINEAR_OK, call, refused

SAVE = ["dtype", "M", "N", "X", "ldx", "Q", "ldq", "S", "lds", "stream"]
RESTORE = ["dtype", "M", "N", "Q", "ldq", "S", "lds", "X", "ldx", "stream"]
SAVE_OK = dict(dtype=0, M=8, N=130, X=FAKE, ldx=130, Q=FAKE, ldq=130, S=FAKE, lds=3, stream=None)
LINEAR8 = ["dtype", "transw", "M", "N", "K", "X", "ldx", "W", "ldw", "bias", "act", "R", "ldr", "Y", "ldy", "Zq", "ldzq",
           "Zs", "ldzs", "stream"]
LINEAR8_OK = dict(LINEAR_OK, Zq=FAKE, ldzq=6, Zs=FAKE, ldzs=1)
BACKWARD8 = ["dtype", "transw", "M", "N", "K", "dY", "lddy", "Zq", "ldzq", "Zs", "ldzs", "act", "Xq", "ldxq", "Xs", "ldxs",
             "W", "ldw", "dX", "lddx", "dW", "lddw", "db", "stream"]
BACKWARD8_OK = dict(BACKWARD_OK, Zq=FAKE, ldzq=6, Zs=FAKE, ldzs=1, Xq=FAKE, ldxq=4, Xs=FAKE, ldxs=1)
LOSS = ["dtype", "transw", "T", "V", "D", "X", "ldx", "W", "ldw", "labels", "loss", "lse", "stream"]
LOSS_OK = dict(dtype=0, transw=1, T=4, V=10, D=8, X=FAKE, ldx=8, W=FAKE, ldw=8, labels=FAKE, loss=FAKE, lse=FAKE + 64,
               stream=None)
GRAD = ["dtype", "transw", "T", "V", "D", "dloss", "incd", "X", "ldx", "W", "ldw", "labels", "lse", "dX", "lddx", "dW", "lddw",
        "stream"]
GRAD_OK = dict(dtype=1, transw=1, T=4, V=10, D=8, dloss=FAKE, incd=1, X=FAKE, ldx=8, W=FAKE, ldw=8, labels=FAKE, lse=FAKE,
               dX=FAKE, lddx=8, dW=FAKE, lddw=8, stream=None)


@pytest.mark.parametrize("name,order", [("sgemm_checkpoint8", SAVE), ("sgemm_restore8", RESTORE)])
@pytest.mark.parametrize("change,why", [
    (dict(dtype=2), "dtype"), (dict(M=-1), "M and N"), (dict(N=-1), "M and N"), (dict(ldx=129), "ldx"),
    (dict(ldq=129), "ldq"), (dict(lds=2), "lds"), (dict(Q=None), "Q or S"), (dict(S=None), "Q or S"), (dict(X=None), "X is NULL"),
    (dict(X=FAKE + 1), "aligned"), (dict(S=FAKE + 2), "aligned"), (dict(M=0, ldq=0), "ldq"),
])
def test_checkpoint_refusals(sgemm_lib, name, order, change, why):
    refused(sgemm_lib, name, order, SAVE_OK, why, **change)
    assert call(sgemm_lib, name, order, SAVE_OK, M=0, X=None, Q=None, S=None) == 0
    assert call(sgemm_lib, name, order, SAVE_OK, N=0, X=None, Q=None, S=None) == 0
    refused(sgemm_lib, name, order, SAVE_OK, "2^31", status=4, M=1 << 31)


@pytest.mark.parametrize("change,why", [
    (dict(dtype=2), "dtype"), (dict(act=5), "activation"), (dict(ldx=3), "ldx"), (dict(ldzq=5), "ldq"), (dict(ldzs=0), "lds"),
    (dict(Zq=None), "Q or S"), (dict(Zs=None), "Q or S"), (dict(Zs=FAKE + 1), "aligned"), (dict(Y=None), "Y is NULL"),
])
def test_linear_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_linear_checkpoint8", LINEAR8, LINEAR8_OK, why, **change)
    assert call(sgemm_lib, "sgemm_linear_checkpoint8", LINEAR8, LINEAR8_OK, M=0, Zq=None, Zs=None) == 0


@pytest.mark.parametrize("change,why", [
    (dict(dtype=7), "dtype"), (dict(act=9), "activation"), (dict(lddy=5), "lddy"), (dict(ldzq=5), "ldq"), (dict(ldxq=3), "ldq"),
    (dict(ldzs=0), "lds"), (dict(ldxs=0), "lds"), (dict(ldw=3), "ldw"), (dict(lddx=3), "lddx"), (dict(lddw=3), "lddw"),
    (dict(dY=None), "dY is NULL"), (dict(Zq=None), "Q or S"), (dict(Xs=None), "Q or S"), (dict(W=None), "W is NULL"),
    (dict(dX=FAKE + 1), "aligned"), (dict(Xs=FAKE + 2), "aligned"), (dict(db=FAKE + 2), "aligned"),
])
def test_backward_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_linear_backward_checkpoint8", BACKWARD8, BACKWARD8_OK, why, **change)


def test_backward_without_outputs_needs_no_device(sgemm_lib):
    nothing = dict(dX=None, dW=None, db=None)
    assert call(sgemm_lib, "sgemm_linear_backward_checkpoint8", BACKWARD8, BACKWARD8_OK, **nothing) == 0
    assert call(sgemm_lib, "sgemm_linear_backward_checkpoint8", BACKWARD8, BACKWARD8_OK, Xq=None, Xs=None, Zq=None,
                Zs=None, ldxq=0, ldzq=6, **nothing) == 0
    assert call(sgemm_lib, "sgemm_linear_backward_checkpoint8", BACKWARD8, BACKWARD8_OK, M=0, dW=None, db=None) == 0
    refused(sgemm_lib, "sgemm_linear_backward_checkpoint8", BACKWARD8, BACKWARD8_OK, "2^31", status=4, M=1 << 31)


HEAD = [(dict(dtype=2), "dtype"), (dict(transw=2), "transw"), (dict(T=-1), "T must"), (dict(V=0), "V and D"),
        (dict(D=0), "V and D"), (dict(ldx=7), "ldx"), (dict(ldw=7), "ldw"), (dict(transw=0, ldw=9, lddw=10), "ldw"),
        (dict(X=None), "X or W"), (dict(W=None), "X or W"), (dict(labels=None), "labels"), (dict(X=FAKE + 1), "aligned"),
        (dict(labels=FAKE + 4), "aligned"), (dict(lse=FAKE + 2), "aligned")]


@pytest.mark.parametrize("change,why", HEAD + [(dict(loss=FAKE + 2), "aligned"), (dict(lse=FAKE), "same array")])
def test_loss_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_cross_entropy", LOSS, LOSS_OK, why, **change)


@pytest.mark.parametrize("change,why", HEAD + [
    (dict(incd=-1), "incd"), (dict(lddx=7), "lddx"), (dict(lddw=7), "lddw"), (dict(transw=0, ldw=10, lddw=9), "lddw"),
    (dict(dloss=None), "dloss"), (dict(lse=None), "dloss or lse"), (dict(dX=FAKE + 1), "aligned"), (dict(dloss=FAKE + 1), "aligned"),
    (dict(T=0, dW=FAKE + 1), "aligned")])
def test_gradient_refusals(sgemm_lib, change, why):
    refused(sgemm_lib, "sgemm_cross_entropy_backward", GRAD, GRAD_OK, why, **change)


def test_head_calls_that_need_no_device(sgemm_lib):
    assert call(sgemm_lib, "sgemm_cross_entropy", LOSS, LOSS_OK, T=0, X=None, labels=None) == 0
    assert call(sgemm_lib, "sgemm_cross_entropy", LOSS, LOSS_OK, loss=None, lse=None) == 0
    assert call(sgemm_lib, "sgemm_cross_entropy_backward", GRAD, GRAD_OK, dX=None, dW=None) == 0
    assert call(sgemm_lib, "sgemm_cross_entropy_backward", GRAD, GRAD_OK, T=0, dW=None) == 0
    refused(sgemm_lib, "sgemm_cross_entropy", LOSS, LOSS_OK, "2^31", status=4, V=1 << 31)
    refused(sgemm_lib, "sgemm_cross_entropy_backward", GRAD, GRAD_OK, "2^31", status=4, T=1 << 31)


def test_python_shapes_and_types(sgemm_lib):
    torch = pytest.importorskip("torch")
    sg = sgemm_lib
    x, w = torch.zeros(3, 8, dtype=torch.bfloat16), torch.zeros(5, 8, dtype=torch.bfloat16)
    labels, f = torch.zeros(3, dtype=torch.int64), torch.zeros(3)
    with pytest.raises(TypeError):  # host tensors
        sg.cross_entropy(x, w, labels)
    with pytest.raises(TypeError):
        sg.checkpoint8(x)
    with pytest.raises(TypeError):
        sg.checkpoint8(x.float())
    with pytest.raises(TypeError):
        sg.cross_entropy(x, w, labels.int())
    with pytest.raises(TypeError):
        sg.cross_entropy_backward(f.bfloat16(), x, w, labels, f)
    for bad in (labels[:2], labels[:, None]):
        with pytest.raises(ValueError):
            sg.cross_entropy(x, w, bad)
    for dloss, lse in ((f[:1], f), (f, f[:2]), (f, torch.zeros(6)[::2])):
        with pytest.raises(ValueError):
            sg.cross_entropy_backward(dloss, x, w, labels, lse)
    for bad in (x[0], x.t()):
        with pytest.raises(ValueError):
            sg.checkpoint8(bad)
    with pytest.raises(ValueError):
        sg.linear(x, w, save_pre="16bit")
    codes, scale = torch.zeros(3, 8, dtype=torch.int8), torch.zeros(3, 1)

    def checkpoint(codes=codes, scale=scale, dtype=torch.bfloat16):
        return sg.Checkpoint8(codes, scale, dtype)

    assert checkpoint().shape == (3, 8) and checkpoint().codes is codes and checkpoint().scale is scale
    for bad in (checkpoint(scale=torch.zeros(3, 2)), checkpoint(scale=f), checkpoint(codes=codes[0]),
                checkpoint(codes=torch.zeros(8, 3, dtype=torch.int8).t())):
        with pytest.raises(ValueError):
            sg.restore8(bad)
    for bad in (checkpoint(codes=codes.to(torch.uint8)), checkpoint(scale=scale.double()), checkpoint(dtype=torch.float32),
                checkpoint()):  # (the last: on the host)
        with pytest.raises(TypeError):
            sg.restore8(bad)
    dy = torch.zeros(3, 5, dtype=torch.bfloat16)
    with pytest.raises(TypeError):  # a checkpoint of another type
        sg.linear_backward(dy, checkpoint(dtype=torch.float16), w)
    with pytest.raises(ValueError):  # of another shape
        sg.linear_backward(dy, checkpoint(codes[:2], scale[:2]), w)
