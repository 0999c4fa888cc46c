"""Host side of the operators around the fused layers: the launches' schedule, and argument checks before
any device is touched (CPU only: no kernel is launched)."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.operators import GatedShape, LossShape, NormShape

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x10000  # aligned fake address: every call below is rejected before any dereference


@pytest.fixture(scope="module")
def L():
    fg.build()
    return fg.lib()


def test_units_are_visited_once_and_evenly(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "units_check")
    subprocess.run([gxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I",
                    os.path.join(ROOT, "backward_optimizer_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "c", "units_check.cpp"), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True)
    assert out.returncode == 0, out.stdout


def _norm(**kw):
    return ctypes.byref(NormShape(**{**dict(T=4, D=64, kind=0, x_type=0, w_type=1, reserved=0), **kw}))


@pytest.mark.parametrize("kw, code", [
    (dict(T=-1), 1), (dict(D=0), 1), (dict(D=2**24 + 1), 1), (dict(kind=2), 1), (dict(x_type=2), 1), (dict(w_type=-1), 1),
    (dict(reserved=1), 1)])
def test_norm_shapes_refused(L, kw, code):
    assert L.forge_layer_norm(A, A, A, A, A, A, 1e-5, _norm(**kw), None) == code
    assert L.forge_layer_norm_backward(A, A, A, A, A, None, A, A, A, A, 1 << 30, _norm(**kw), None) == code
    assert L.forge_layer_norm_backward_workspace(_norm(**kw)) == -1


def test_norm_arguments_refused(L):
    nan = float("nan")
    for args, code in (((None, A, A, A, A, A, 1e-5), 1), ((A, None, A, A, A, A, 1e-5), 1), ((A, A, A, None, A, A, 1e-5), 1),
                       ((A, A, A, A, A, A, nan), 1), ((A, A, A, A, A, A, -1.0), 1), ((A + 1, A, A, A, A, A, 1e-5), 3),
                       ((A, A + 2, A, A, A, A, 1e-5), 3), ((A, A, A, A, A + 2, A, 1e-5), 3)):
        assert L.forge_layer_norm(*args, _norm(), None) == code
    assert L.forge_layer_norm(A, A, A, A, A, A, 1e-5, None, None) == 1
    assert L.forge_layer_norm(A, A, A, A, None, A, 1e-5, _norm(kind=1), None) == 1  # an RMS norm with a bias
    assert L.forge_layer_norm(A, A, A, A, A, A, 1e-5, _norm(T=0), None) == 0
    for i in (0, 1, 2, 3, 4, 6, 7, 8):  # dy, x, weight, mean, rstd, (add may be null), dx, dweight, dbias
        args = [A] * 9
        args[i] = None
        assert L.forge_layer_norm_backward(*args, A, 1 << 30, _norm(), None) == 1


def _gated(**kw):
    return ctypes.byref(GatedShape(**{**dict(T=4, d_model=64, d_ff=128, act=0, reserved=0), **kw}))


@pytest.mark.parametrize("kw", [dict(T=-1), dict(d_model=0), dict(d_model=60), dict(d_ff=4), dict(d_ff=2**31), dict(act=3),
                                dict(act=-1), dict(reserved=1), dict(T=2**30, d_ff=2**20)])
def test_gated_shapes_refused(L, kw):
    hp = fg.hparams_struct()
    layer = fg.ForgeLayer(None, None, A, A, A, None, 0, 0, 0, 0)
    assert L.forge_gated_mlp(A, A, A, A, A, A, A, A, A, 1 << 40, _gated(**kw), None) == 1
    assert L.forge_gated_mlp_backward(*[A] * 12, 1 << 40, _gated(**kw), None) == 1
    assert L.forge_gated_mlp_backward_step(A, A, A, A, *[ctypes.byref(layer)] * 3, A, A, 1 << 40, 0, 0, ctypes.byref(hp),
                                           _gated(**kw), 1, None) == 1
    assert L.forge_gated_mlp_workspace(_gated(**kw), 0) == -1


def test_gated_arguments_refused(L):
    for i in (0, 1, 2, 3, 5):  # X, Wg, Wu, Wd, Y; the residual may be null
        args = [A] * 8
        args[i] = None
        assert L.forge_gated_mlp(*args, A, 1 << 40, _gated(), None) == 1
        args[i] = A + 16
        assert L.forge_gated_mlp(*args, A, 1 << 40, _gated(), None) == 3
    assert L.forge_gated_mlp(A, A, A, A, None, A, A, None, A, 1 << 40, _gated(), None) == 1  # G without U
    assert L.forge_gated_mlp(A, A, A, A, None, A, A, A, None, 0, _gated(T=0), None) == 0
    for i in (0, 1, 2, 3, 4, 5, 6, 8, 9, 10):  # all but dX
        args = [A] * 11
        args[i] = None
        assert L.forge_gated_mlp_backward(*args, A, 1 << 40, _gated(), None) == 1
    hp = ctypes.byref(fg.hparams_struct())
    good = fg.ForgeLayer(None, None, A, A, A, None, 0, 0, 0, 0)
    for field, code in (("W", 1), ("m", 1), ("v", 1)):
        bad = fg.ForgeLayer(None, None, A, A, A, None, 0, 0, 0, 0)
        setattr(bad, field, None)
        for i in range(3):
            layers = [ctypes.byref(bad if i == j else good) for j in range(3)]
            assert L.forge_gated_mlp_backward_step(A, A, A, A, *layers, A, A, 1 << 40, 0, 0, hp, _gated(), 1, None) == code
    layers = [ctypes.byref(good)] * 3
    assert L.forge_gated_mlp_backward_step(A, A, A, A, *layers, A, A, 1 << 40, 5, 0, hp, _gated(), 1, None) == 1  # state
    assert L.forge_gated_mlp_backward_step(A, A, A, A, *layers, A, A, 1 << 40, 0, 9, hp, _gated(), 1, None) == 1  # optimizer
    assert L.forge_gated_mlp_backward_step(A, A, A, A, *layers, A, A, 1 << 40, 0, 0, hp, _gated(), 0, None) == 1  # step
    assert L.forge_gated_mlp_backward_step(A, A, A, A, None, *layers[1:], A, A, 1 << 40, 0, 0, hp, _gated(), 1, None) == 1
    assert L.forge_gated_mlp_backward_step(A, A, A, A, *layers, A + 2, A, 1 << 40, 0, 0, hp, _gated(), 1, None) == 3


def _loss(**kw):
    return ctypes.byref(LossShape(**{**dict(T=4, vocab=100, d_model=64, ignore_index=-100, reserved=0), **kw}))


@pytest.mark.parametrize("kw", [dict(T=-1), dict(vocab=0), dict(vocab=2**31), dict(d_model=0), dict(d_model=12),
                                dict(reserved=1), dict(T=2**30, vocab=2**20)])
def test_loss_shapes_refused(L, kw):
    hp = ctypes.byref(fg.hparams_struct())
    assert L.forge_linear_cross_entropy(A, A, A, A, A, A, 1 << 40, _loss(**kw), None) == 1
    assert L.forge_linear_cross_entropy_backward(*[A] * 8, 1 << 40, _loss(**kw), None) == 1
    assert L.forge_linear_cross_entropy_step(A, A, A, A, A, A, A, A, None, A, 1 << 40, 0, 0, hp, _loss(**kw), 1, 0, None) == 1
    assert L.forge_linear_cross_entropy_workspace(_loss(**kw), 1) == -1


def test_loss_arguments_refused(L):
    hp = ctypes.byref(fg.hparams_struct())
    for i in range(5):
        args = [A] * 5
        args[i] = None
        assert L.forge_linear_cross_entropy(*args, A, 1 << 40, _loss(), None) == 1
        args[i] = A + 2
        assert L.forge_linear_cross_entropy(*args, A, 1 << 40, _loss(), None) == 3
    for i in range(5):  # X, W, target, lse, dloss
        args = [A] * 7
        args[i] = None
        assert L.forge_linear_cross_entropy_backward(*args, A, 1 << 40, _loss(), None) == 1
    assert L.forge_linear_cross_entropy_backward(A, A, A, A, A, None, None, A, 1 << 40, _loss(), None) == 1
    assert L.forge_linear_cross_entropy_backward(A, A, A, A, A, A + 8, A, A, 1 << 40, _loss(), None) == 3
    for bad in (dict(m=None), dict(v=None), dict(W=None)):
        a = {**dict(W=A, m=A, v=A), **bad}
        assert L.forge_linear_cross_entropy_step(A, a["W"], A, A, A, A, a["m"], a["v"], None, A, 1 << 40, 0, 0, hp, _loss(), 1,
                                                 0, None) == 1
    # INT8 states need their scales, and blocks of 64 within a row
    assert L.forge_linear_cross_entropy_step(A, A, A, A, A, A, A, A, None, A, 1 << 40, 1, 0, hp, _loss(), 1, 0, None) == 1
    assert L.forge_linear_cross_entropy_step(A, A, A, A, A, A, A, A, A, A, 1 << 40, 1, 0, hp, _loss(d_model=72), 1, 0, None) == 1


def test_cpu_tensors_refused():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        fg.layer_norm(x, w, None, x.clone())
    with pytest.raises(ValueError, match="CUDA"):
        fg.gated_mlp(x, x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        fg.linear_cross_entropy(x, x, torch.zeros(4, dtype=torch.int64), w, w)
