"""Refusals of the operators' launch-shape queries (CPU only)."""
import ctypes

import pytest

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300 import operators as ops


def test_refusals():
    fg.build()
    L = fg.lib()
    out = [ctypes.c_int32() for _ in range(4)]
    p = [ctypes.byref(o) for o in out]
    good, bad = ops.GatedShape(4, 64, 128, 0, 0), ops.GatedShape(4, 60, 128, 0, 0)
    for shape, launch in ((bad, 0), (good, -1), (good, 4)):
        assert L.forge_gated_mlp_launch_shape(ctypes.byref(shape), launch, *p) == 1
    good, bad = ops.LossShape(4, 100, 64, -100, 0), ops.LossShape(4, 0, 64, -100, 0)
    for shape, launch in ((bad, 0), (good, -1), (good, 3)):
        assert L.forge_linear_cross_entropy_launch_shape(ctypes.byref(shape), launch, *p) == 1
    assert L.forge_linear_cross_entropy_launch_shape(ctypes.byref(good), 0, None, *p[1:]) == 1
    with pytest.raises(ValueError):
        ops.gated_launch_shape(4, 64, 128, "g")
    with pytest.raises(ValueError):
        ops.loss_launch_shape(4, 100, 64, "up")
