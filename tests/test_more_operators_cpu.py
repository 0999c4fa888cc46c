"""Argument checks of the products grouped by expert, dropout and the preference loss, before any device is touched
(CPU only: no kernel is launched)."""
import ctypes

import pytest
import torch

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.operators import ExpertGatedShape, ExpertLinearShape, PreferenceShape

A = 0x10000  # aligned fake address: every call below is rejected before any dereference
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    fg.build()
    return fg.lib()


def _linear(**kw):
    return ctypes.byref(ExpertLinearShape(**{**dict(rows=4, experts=2, d_in=64, d_out=128, reserved=0), **kw}))


def _gated(**kw):
    return ctypes.byref(ExpertGatedShape(**{**dict(rows=4, experts=2, d_model=64, d_ff=128, act=0, reserved=0), **kw}))


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(rows=2**31), dict(experts=0), dict(experts=1025), dict(d_in=0),
                                dict(d_in=60), dict(d_out=4), dict(d_out=2**31), dict(reserved=1), dict(rows=2**30, d_out=2**20)])
def test_linear_shapes_refused(L, kw):
    assert L.forge_expert_linear(A, A, A, A, A, BIG, _linear(**kw), None) == 1
    assert L.forge_expert_linear_backward(A, A, A, A, A, A, A, BIG, _linear(**kw), None) == 1
    assert L.forge_expert_linear_workspace(_linear(**kw), 0) == -1


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(experts=0), dict(experts=1025), dict(d_model=0), dict(d_model=60),
                                dict(d_ff=4), dict(act=3), dict(act=-1), dict(reserved=1), dict(rows=2**30, d_ff=2**20)])
def test_gated_shapes_refused(L, kw):
    assert L.forge_expert_gated_mlp(*[A] * 9, BIG, _gated(**kw), None) == 1
    assert L.forge_expert_gated_mlp_backward(*[A] * 13, BIG, _gated(**kw), None) == 1
    assert L.forge_expert_gated_mlp_workspace(_gated(**kw), 0) == -1
    assert L.forge_expert_gated_mlp_workspace(_gated(**kw), 1) == -1


def _each(n, skip=()):
    """Argument lists with one of n addresses missing, and with one misaligned."""
    for i in range(n):
        if i not in skip:
            yield [None if j == i else A for j in range(n)], 1


def test_expert_arguments_refused(L):
    for args, code in _each(4):
        assert L.forge_expert_linear(*args, A, BIG, _linear(), None) == code
    for i, off in ((0, 16), (1, 16), (3, 16), (2, 2)):  # X, W, Y; offsets
        args = [A + off if j == i else A for j in range(4)]
        assert L.forge_expert_linear(*args, A, BIG, _linear(), None) == 3
    for args, code in _each(6, skip=(4, 5)):
        assert L.forge_expert_linear_backward(*args, A, BIG, _linear(), None) == code
    assert L.forge_expert_linear_backward(A, A, A, A, None, None, A, BIG, _linear(), None) == 1
    assert L.forge_expert_linear_backward(A, A, A, A, A + 8, None, A, BIG, _linear(), None) == 3
    for args, code in _each(6):  # X, Wg, Wu, Wd, offsets, Y
        assert L.forge_expert_gated_mlp(*args, A, A, A, BIG, _gated(), None) == code
    assert L.forge_expert_gated_mlp(*[A] * 6, A, None, A, BIG, _gated(), None) == 1  # G without U
    assert L.forge_expert_gated_mlp(*[A] * 6, A, A + 8, A, BIG, _gated(), None) == 3
    for args, code in _each(12, skip=(8,)):  # dX may be null
        assert L.forge_expert_gated_mlp_backward(*args, A, BIG, _gated(), None) == code
    assert L.forge_expert_linear(None, None, None, None, None, 0, _linear(rows=0), None) == 0
    assert L.forge_expert_gated_mlp(*[None] * 9, 0, _gated(rows=0), None) == 0
    for f, n in ((L.forge_expert_linear, 4), (L.forge_expert_gated_mlp, 8)):
        assert f(*[A] * n, A, BIG, None, None) == 1


def test_dropout_refused(L):
    def call(x=A, r=None, y=A, n=8, t=0, p=0.1, at=None):
        return L.forge_dropout(x, r, y, n, t, p, 0, 0, at, None)
    for kw in (dict(x=None), dict(y=None), dict(n=-1), dict(n=2**43), dict(t=2), dict(t=-1), dict(p=-0.1), dict(p=1.01),
               dict(p=float("nan"))):
        assert call(**kw) == 1, kw
    for kw in (dict(x=A + 1), dict(y=A + 1), dict(r=A + 1), dict(t=1, x=A + 2), dict(at=A + 4)):
        assert call(**kw) == 3, kw
    assert call(x=None, y=None, n=0) == 0


def _pref(**kw):
    return ctypes.byref(PreferenceShape(**{**dict(tokens=9, pairs=2, kind=0, mean=0, beta=0.1, smoothing=0.0, margin=0.0,
                                                  reserved=0), **kw}))


@pytest.mark.parametrize("kw", [dict(tokens=-1), dict(tokens=2**30 + 1), dict(pairs=-1), dict(pairs=2**24 + 1), dict(kind=3),
                                dict(kind=-1), dict(beta=0.0), dict(beta=-1.0), dict(beta=float("inf")), dict(beta=float("nan")),
                                dict(smoothing=-0.1), dict(smoothing=1.0), dict(smoothing=float("nan")),
                                dict(kind=1, smoothing=0.1), dict(margin=float("nan")), dict(reserved=1)])
def test_preference_shapes_refused(L, kw):
    assert L.forge_preference_loss(*[A] * 8, BIG, _pref(**kw), None) == 1
    assert L.forge_preference_loss_backward(*[A] * 5, _pref(**kw), None) == 1
    assert L.forge_preference_loss_workspace(_pref(**kw)) == -1


def test_preference_arguments_refused(L):
    for i in (0, 3, 4, 7):  # nll, offsets, loss, workspace; ref, mask, reward and slope may be null
        args = [None if j == i else A for j in range(8)]
        assert L.forge_preference_loss(*args, BIG, _pref(), None) == 1
    for i in (0, 1, 3, 4, 5, 6):
        args = [A + 2 if j == i else A for j in range(8)]
        assert L.forge_preference_loss(*args, BIG, _pref(), None) == 3
    need = L.forge_preference_loss_workspace(_pref())
    assert need > 0
    assert L.forge_preference_loss(*[A] * 8, need - 1, _pref(), None) == 1
    assert L.forge_preference_loss(*[A] * 7, A + 16, BIG, _pref(), None) == 3
    for i in (0, 1, 3, 4):  # dloss, slope, offsets, dnll
        args = [None if j == i else A for j in range(5)]
        assert L.forge_preference_loss_backward(*args, _pref(), None) == 1
        args = [A + 1 if j == i else A for j in range(5)]
        assert L.forge_preference_loss_backward(*args, _pref(), None) == 3
    assert L.forge_preference_loss(*[None] * 8, 0, _pref(pairs=0), None) == 0
    assert L.forge_preference_loss_backward(*[None] * 5, _pref(tokens=0), None) == 0


def test_tensors_on_the_host_are_refused(L):
    x, w = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(2, 8, 8, dtype=torch.bfloat16)
    off = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fg.expert_linear(x, w, off, x)
    with pytest.raises(ValueError):
        fg.expert_gated_mlp(x, w, w, w, off, x)
    with pytest.raises(ValueError):
        fg.dropout(x, x, 0.5)
    with pytest.raises(ValueError):
        fg.preference_loss(torch.zeros(4), None, off, torch.zeros(1))
