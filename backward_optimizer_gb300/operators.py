"""The operators around the fused layers: the norm, the gated feed-forward block, the cross entropy of a
linear head, linear layers and gated blocks with a weight for each expert, dropout from a counter, and the
preference loss of pairs of sequences, each with its backward pass.

Like the rest of the binding this module checks and marshals arguments; the computation is the
library's.  Results are written to the tensors passed for them.  Tensors are contiguous and on the
current device.  Workspace comes from PyTorch's allocator, for the stream that the call runs on.  Calls on
the current stream that need up to 16 MiB of it keep it from call to call, one buffer per host thread and
stream until the thread ends, from the memory pool that was in use when it was made.
`include/forge.h` documents every operator's formulas, types and special cases.
"""
from __future__ import annotations

import ctypes
import threading
from typing import Any

import torch

import backward_optimizer_gb300 as _fg

NORM_KINDS = {"layer": 0, "rms": 1}
PREFERENCES = {"sigmoid": 0, "hinge": 1, "ipo": 2}
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1, "relu": 2}
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_BF16, _F32 = torch.bfloat16, torch.float32


class NormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("kind", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("w_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GatedShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int64), ("d_ff", ctypes.c_int64), ("act", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class LossShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("vocab", ctypes.c_int64), ("d_model", ctypes.c_int64),
                ("ignore_index", ctypes.c_int64), ("reserved", ctypes.c_int64)]


class PreferenceShape(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("pairs", ctypes.c_int64), ("kind", ctypes.c_int32), ("mean", ctypes.c_int32),
                ("beta", ctypes.c_float), ("smoothing", ctypes.c_float), ("margin", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class ExpertLinearShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("experts", ctypes.c_int64), ("d_in", ctypes.c_int64), ("d_out", ctypes.c_int64),
                ("reserved", ctypes.c_int64)]


class ExpertGatedShape(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("experts", ctypes.c_int64), ("d_model", ctypes.c_int64), ("d_ff", ctypes.c_int64),
                ("act", ctypes.c_int32), ("reserved", ctypes.c_int32)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the library's functions that this module calls."""
    vp, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float
    norm, gated, loss = (ctypes.POINTER(t) for t in (NormShape, GatedShape, LossShape))
    elinear, egated, pref = (ctypes.POINTER(t) for t in (ExpertLinearShape, ExpertGatedShape, PreferenceShape))
    layer, hp = ctypes.POINTER(_fg.ForgeLayer), ctypes.POINTER(_fg.ForgeHparams)
    for name, args in {
        "forge_layer_norm": [vp] * 6 + [f32, norm, vp],
        "forge_layer_norm_backward": [vp] * 10 + [i64, norm, vp],
        "forge_gated_mlp": [vp] * 9 + [i64, gated, vp],
        "forge_gated_mlp_backward": [vp] * 12 + [i64, gated, vp],
        "forge_gated_mlp_backward_step": [vp] * 4 + [layer] * 3 + [vp, vp, i64, i32, ctypes.c_int, hp, gated, i64, vp],
        "forge_linear_cross_entropy": [vp] * 6 + [i64, loss, vp],
        "forge_linear_cross_entropy_backward": [vp] * 8 + [i64, loss, vp],
        "forge_linear_cross_entropy_step": [vp] * 10 + [i64, i32, ctypes.c_int, hp, loss, i64, u64, vp],
        "forge_expert_linear": [vp] * 5 + [i64, elinear, vp],
        "forge_expert_linear_backward": [vp] * 7 + [i64, elinear, vp],
        "forge_expert_gated_mlp": [vp] * 9 + [i64, egated, vp],
        "forge_expert_gated_mlp_backward": [vp] * 13 + [i64, egated, vp],
        "forge_expert_linear_backward_step": [vp] * 9 + [i64, i32, ctypes.c_int, hp, elinear, i64, u64, vp],
        "forge_expert_gated_mlp_backward_step": [vp] * 4 + [layer] * 3 + [vp] * 3 + [i64, i32, ctypes.c_int, hp, egated, i64, vp],
        "forge_dropout": [vp] * 3 + [i64, i32, ctypes.c_double, u64, u64, vp, vp],
        "forge_preference_loss": [vp] * 8 + [i64, pref, vp],
        "forge_preference_loss_backward": [vp] * 5 + [pref, vp],
        "forge_gated_mlp_launch_shape": [gated, i32] + [ctypes.POINTER(i32)] * 4,
        "forge_linear_cross_entropy_launch_shape": [loss, i32] + [ctypes.POINTER(i32)] * 4,
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, ctypes.c_int
    for name, args in {
        "forge_layer_norm_backward_workspace": [norm],
        "forge_gated_mlp_workspace": [gated, i32],
        "forge_linear_cross_entropy_workspace": [loss, i32],
        "forge_expert_linear_workspace": [elinear, i32],
        "forge_preference_loss_workspace": [pref],
        "forge_expert_gated_mlp_workspace": [egated, i32],
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, i64


# The C structure of a shape, ready to pass, and the workspace that the shape needs, by sizes: a training
# loop makes the same calls over and over, and building them costs as much host time as a small kernel.
_shapes: dict = {}


class _Shape:
    __slots__ = ("arg", "bytes")

    def __init__(self, struct):
        self.arg, self.bytes = ctypes.byref(struct), {}  # workspace bytes by device and direction


def _shape(cls, *values) -> _Shape:
    key = (cls, values)
    s = _shapes.get(key)
    if s is None:
        if len(_shapes) >= 4096:
            _shapes.clear()
        s = _shapes[key] = _Shape(cls(*values))
    return s


# Small workspaces are kept, one per host thread and stream: calls of one thread on one stream use them one
# after another, and asking PyTorch's allocator costs as much host time as a small call's kernels take.
# Captured calls take theirs from the graph's own pool, since a graph runs on streams of its own choosing.
_KEEP = 16 << 20
_kept = threading.local()


def _workspace(shape: _Shape, name: str, dev: int, stream, raw: int, *more):
    """Pointer and size of a workspace at least as large as `name` answers for the shape, and the tensor
    that holds it."""
    n = shape.bytes.get((dev, more))
    if n is None:
        n = getattr(_fg.lib(), name)(shape.arg, *more)
        if n >= 0:  # else the call itself says what is wrong
            shape.bytes[(dev, more)] = n
    if n <= 0:
        return _NONE
    if stream is None:
        if n > _KEEP or torch._C._cuda_isCurrentStreamCapturing():
            t = torch.empty(n, dtype=torch.uint8, device=dev)
            return t.data_ptr(), n, t
        try:
            kept = _kept.by_stream
        except AttributeError:
            kept = _kept.by_stream = {}
        w = kept.get((dev, raw))
        if w is None or w[1] < n:
            size = min(_KEEP, max(2 * n, 1 << 20))
            t = torch.empty(size, dtype=torch.uint8, device=dev)
            w = kept[(dev, raw)] = (t.data_ptr(), size, t)
        return w
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(raw)
    with torch.cuda.stream(s):
        t = torch.empty(n, dtype=torch.uint8, device=dev)
    return t.data_ptr(), n, t


_NONE = (None, 0, None)


def _device(x) -> int:
    """The current device's number; x is checked to be there."""
    if not x.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    dev = x.get_device()
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors on {x.device}, but the current device is cuda:{torch.cuda.current_device()}")
    return dev


def _raw_stream(stream, dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _fg._stream(stream)


def _take(t, dtype, shape: tuple, dev: int, name: str):
    """The address of an argument, checked: its type, shape, device and layout.  None stays None."""
    if t is None:
        return None
    if t.dtype is not dtype:
        raise TypeError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    if t.get_device() != dev:
        raise ValueError(f"{name}: on {t.device}, expected cuda:{dev}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous (row-major)")
    return t.data_ptr()


def _one_of(table: dict, key: str, name: str) -> int:
    v = table.get(key)
    if v is None:
        raise ValueError(f"{name}: {key!r}, expected one of {list(table)}")
    return v


def _type(t, name: str) -> int:
    v = _TYPES.get(t.dtype)
    if v is None:
        raise TypeError(f"{name}: dtype {t.dtype}, expected one of {[str(d) for d in _TYPES]}")
    return v


def _matrix(t, name: str) -> tuple:
    if t.dim() != 2:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected 2")
    return tuple(t.shape)


def _vector(t, name: str) -> int:
    if t.dim() != 1:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected 1")
    return t.shape[0]


def _states(dev: int, W, m, v, qscales) -> None:
    _fg._state_args(W, m, v, qscales)
    for t, name in ((m, "m"), (v, "v"), (qscales, "qscales")):
        if t is not None:
            _take(t, t.dtype, tuple(t.shape), dev, name)


# ------------------------------------------------------------------ norm


def layer_norm(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5, kind: str = "layer", stream=None) -> None:
    """y [T, D] = norm(x) * weight (+ bias) row by row: the layer norm, or with kind="rms" the RMS norm
    (no mean, no bias).  x and y bf16 or FP32, weight and bias [D] bf16 or FP32.  mean and rstd, FP32 [T],
    are what layer_norm_backward needs."""
    dev = _device(x)
    T, D = rows = _matrix(x, "x")
    dt, wt = x.dtype, weight.dtype
    shape = _shape(NormShape, T, D, _one_of(NORM_KINDS, kind, "kind"), _type(x, "x"), _type(weight, "weight"), 0)
    st = _fg.lib().forge_layer_norm(
        _take(x, dt, rows, dev, "x"), _take(weight, wt, (D,), dev, "weight"), _take(bias, wt, (D,), dev, "bias"),
        _take(y, dt, rows, dev, "y"), _take(mean, _F32, (T,), dev, "mean"), _take(rstd, _F32, (T,), dev, "rstd"), eps,
        shape.arg, _raw_stream(stream, dev))
    _fg._check(st, "forge_layer_norm")


def layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias=None, add=None, kind: str = "layer",
                        stream=None) -> None:
    """dx [T, D], dweight and dbias (FP32 [D]) of layer_norm from its x and its mean and rstd (RMS norm:
    mean and dbias None).  add [T, D], the gradient along a residual branch past the norm, is added to dx."""
    dev = _device(x)
    T, D = rows = _matrix(x, "x")
    dt = x.dtype
    shape = _shape(NormShape, T, D, _one_of(NORM_KINDS, kind, "kind"), _type(x, "x"), _type(weight, "weight"), 0)
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_layer_norm_backward_workspace", dev, stream, raw)
    st = _fg.lib().forge_layer_norm_backward(
        _take(dy, dt, rows, dev, "dy"), _take(x, dt, rows, dev, "x"),
        _take(weight, weight.dtype, (D,), dev, "weight"), _take(mean, _F32, (T,), dev, "mean"),
        _take(rstd, _F32, (T,), dev, "rstd"), _take(add, dt, rows, dev, "add"), _take(dx, dt, rows, dev, "dx"),
        _take(dweight, _F32, (D,), dev, "dweight"), _take(dbias, _F32, (D,), dev, "dbias"), ws, n, shape.arg,
        raw)
    _fg._check(st, "forge_layer_norm_backward")


# ------------------------------------------------------------------ gated feed-forward block


def gated_mlp(X, Wg, Wu, Wd, Y, G=None, U=None, residual=None, act: str = "silu", stream=None) -> None:
    """Y [T, D] = (act(X Wg^T) * (X Wu^T)) Wd^T (+ residual), everything bf16: X [T, D], Wg and Wu [F, D],
    Wd [D, F].  G and U [T, F], both or neither: X Wg^T and X Wu^T, which the backward pass needs."""
    dev = _device(X)
    (T, D), F = _matrix(X, "X"), _matrix(Wg, "Wg")[0]
    shape = _shape(GatedShape, T, D, F, _one_of(ACTIVATIONS, act, "act"), 0)
    x, wg, wu = _take(X, _BF16, (T, D), dev, "X"), _take(Wg, _BF16, (F, D), dev, "Wg"), _take(Wu, _BF16, (F, D), dev, "Wu")
    wd, y, r = _take(Wd, _BF16, (D, F), dev, "Wd"), _take(Y, _BF16, (T, D), dev, "Y"), _take(residual, _BF16, (T, D), dev, "residual")
    g, u = _take(G, _BF16, (T, F), dev, "G"), _take(U, _BF16, (T, F), dev, "U")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_gated_mlp_workspace", dev, stream, raw, 0)
    _fg._check(_fg.lib().forge_gated_mlp(x, wg, wu, wd, r, y, g, u, ws, n, shape.arg, raw),
               "forge_gated_mlp")


def gated_mlp_backward(dY, X, G, U, Wg, Wu, Wd, dX, dWg, dWu, dWd, act: str = "silu", stream=None) -> None:
    """The block's gradients, bf16, from dY [T, D] and the forward pass's X, G and U.  dX may be None."""
    dev = _device(X)
    (T, D), F = _matrix(X, "X"), _matrix(Wg, "Wg")[0]
    shape = _shape(GatedShape, T, D, F, _one_of(ACTIVATIONS, act, "act"), 0)
    args = [_take(t, _BF16, s, dev, name) for t, s, name in (
        (dY, (T, D), "dY"), (X, (T, D), "X"), (G, (T, F), "G"), (U, (T, F), "U"), (Wg, (F, D), "Wg"), (Wu, (F, D), "Wu"),
        (Wd, (D, F), "Wd"), (dX, (T, D), "dX"), (dWg, (F, D), "dWg"), (dWu, (F, D), "dWu"), (dWd, (D, F), "dWd"))]
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_gated_mlp_workspace", dev, stream, raw, 1)
    _fg._check(_fg.lib().forge_gated_mlp_backward(*args, ws, n, shape.arg, raw),
               "forge_gated_mlp_backward")


def gated_mlp_backward_step(dY, X, G, U, gate, up, down, dX=None, act: str = "silu", opt: str = "adamw", hp: Any = None,
                            step: int = 1, stream=None) -> None:
    """The block's backward pass with the fused step: dX (None: not computed) from the weights as they are,
    then W, m, v of the three layers updated in place.  gate, up and down are (W, m, v, qscales, seed), as
    fused_dw_step takes them, all with the same state format."""
    dev = _device(X)
    (T, D), F = _matrix(X, "X"), _matrix(gate[0], "gate's W")[0]
    shape = _shape(GatedShape, T, D, F, _one_of(ACTIVATIONS, act, "act"), 0)
    args = [_take(t, _BF16, s, dev, name) for t, s, name in (
        (dY, (T, D), "dY"), (X, (T, D), "X"), (G, (T, F), "G"), (U, (T, F), "U"))]
    layers, states, p = [], set(), _fg._ptr
    for (W, m, v, q, seed), s, name in ((gate, (F, D), "gate"), (up, (F, D), "up"), (down, (D, F), "down")):
        w = _take(W, _BF16, s, dev, f"{name}'s W")
        _states(dev, W, m, v, q)
        states.add(_fg._state_of(m, v))
        layers.append(_fg.ForgeLayer(None, None, w, p(m), p(v), p(q), 0, 0, 0, int(seed) & (2**64 - 1)))
    if len(states) > 1:
        raise TypeError("the three layers must use the same state format")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_gated_mlp_workspace", dev, stream, raw, 1)
    st = _fg.lib().forge_gated_mlp_backward_step(
        *args, *(ctypes.byref(a) for a in layers), _take(dX, _BF16, (T, D), dev, "dX"), ws, n, states.pop(),
        _fg.OPT_KINDS[opt], _fg._hp_arg(hp), shape.arg, int(step), raw)
    _fg._check(st, "forge_gated_mlp_backward_step")


# ------------------------------------------------------------------ cross entropy of a linear head


def linear_cross_entropy(X, W, target, loss, lse, ignore_index: int = -100, stream=None) -> None:
    """loss [T] = lse - logit of the target, lse [T] = log sum exp of the logits X W^T (both FP32), without
    the logits in memory: X [T, D] and W [V, D] bf16, target [T] int64.  The loss is 0 where the target is
    ignore_index, NaN at any other target outside 0 .. V-1."""
    dev = _device(X)
    (T, D), V = _matrix(X, "X"), _matrix(W, "W")[0]
    shape = _shape(LossShape, T, V, D, int(ignore_index), 0)
    x, w, t = _take(X, _BF16, (T, D), dev, "X"), _take(W, _BF16, (V, D), dev, "W"), _take(target, torch.int64, (T,), dev, "target")
    out, l = _take(loss, _F32, (T,), dev, "loss"), _take(lse, _F32, (T,), dev, "lse")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_linear_cross_entropy_workspace", dev, stream, raw, 0)
    _fg._check(_fg.lib().forge_linear_cross_entropy(x, w, t, out, l, ws, n, shape.arg, raw),
               "forge_linear_cross_entropy")


def _loss_gradient_args(X, W, target, lse, dloss, ignore_index: int):
    dev = _device(X)
    (T, D), V = _matrix(X, "X"), _matrix(W, "W")[0]
    return dev, T, D, V, _shape(LossShape, T, V, D, int(ignore_index), 0), [
        _take(X, _BF16, (T, D), dev, "X"), _take(W, _BF16, (V, D), dev, "W"), _take(target, torch.int64, (T,), dev, "target"),
        _take(lse, _F32, (T,), dev, "lse"), _take(dloss, _F32, (T,), dev, "dloss")]


def linear_cross_entropy_backward(X, W, target, lse, dloss, dX, dW, ignore_index: int = -100, stream=None) -> None:
    """dX [T, D] and dW [V, D] (bf16, either may be None) given dloss [T], the gradient of each token's loss,
    and the forward pass's lse."""
    dev, T, D, V, shape, args = _loss_gradient_args(X, W, target, lse, dloss, ignore_index)
    dx, dw = _take(dX, _BF16, (T, D), dev, "dX"), _take(dW, _BF16, (V, D), dev, "dW")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_linear_cross_entropy_workspace", dev, stream, raw, 1)
    st = _fg.lib().forge_linear_cross_entropy_backward(*args, dx, dw, ws, n, shape.arg, raw)
    _fg._check(st, "forge_linear_cross_entropy_backward")


def linear_cross_entropy_step(X, W, target, lse, dloss, dX=None, m=None, v=None, qscales=None, ignore_index: int = -100,
                              opt: str = "adamw", hp: Any = None, step: int = 1, seed: int = 0, stream=None) -> None:
    """The same backward pass with the fused step in place of dW: dX (None: not computed) from the weights as
    they are, and W, m, v updated in place, as fused_dw_step takes them."""
    dev, T, D, V, shape, args = _loss_gradient_args(X, W, target, lse, dloss, ignore_index)
    dx, p = _take(dX, _BF16, (T, D), dev, "dX"), _fg._ptr
    _states(dev, W, m, v, qscales)
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_linear_cross_entropy_workspace", dev, stream, raw, 1)
    st = _fg.lib().forge_linear_cross_entropy_step(
        *args, dx, p(m), p(v), p(qscales), ws, n, _fg._state_of(m, v), _fg.OPT_KINDS[opt], _fg._hp_arg(hp), shape.arg,
        int(step), int(seed) & (2**64 - 1), raw)
    _fg._check(st, "forge_linear_cross_entropy_step")


# ------------------------------------------------------------------ products grouped by expert


def _grouped(X, W, name: str):
    """Device, rows, width, experts and the weight's other width."""
    dev = _device(X)
    R, D = _matrix(X, "X")
    if W.dim() != 3:
        raise ValueError(f"{name}: {W.dim()} dimensions, expected 3")
    return dev, R, D, W.shape[0], W.shape[1]


def expert_linear(X, W, offsets, Y, stream=None) -> None:
    """Y[r] = X[r] W[e]^T for the rows r = offsets[e] .. offsets[e+1]-1 of each expert e, everything bf16: X [R, d_in]
    sorted by expert, W [E, d_out, d_in], Y [R, d_out]; offsets int32 [E+1] on the device, never read on the host.
    Rows of no expert are left as they were."""
    dev, R, D, E, F = _grouped(X, W, "W")
    shape = _shape(ExpertLinearShape, R, E, D, F, 0)
    x, w = _take(X, _BF16, (R, D), dev, "X"), _take(W, _BF16, (E, F, D), dev, "W")
    o, y = _take(offsets, torch.int32, (E + 1,), dev, "offsets"), _take(Y, _BF16, (R, F), dev, "Y")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_expert_linear_workspace", dev, stream, raw, 0)
    _fg._check(_fg.lib().forge_expert_linear(x, w, o, y, ws, n, shape.arg, raw), "forge_expert_linear")


def expert_linear_backward(dY, X, W, offsets, dX, dW, stream=None) -> None:
    """dX [R, d_in] and dW [E, d_out, d_in] (bf16, either may be None) of expert_linear from dY [R, d_out].  dW of an
    expert without rows is zero."""
    dev, R, D, E, F = _grouped(X, W, "W")
    shape = _shape(ExpertLinearShape, R, E, D, F, 0)
    args = [_take(t, dt, s, dev, name) for t, dt, s, name in (
        (dY, _BF16, (R, F), "dY"), (X, _BF16, (R, D), "X"), (W, _BF16, (E, F, D), "W"),
        (offsets, torch.int32, (E + 1,), "offsets"), (dX, _BF16, (R, D), "dX"), (dW, _BF16, (E, F, D), "dW"))]
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_expert_linear_workspace", dev, stream, raw, 1)
    _fg._check(_fg.lib().forge_expert_linear_backward(*args, ws, n, shape.arg, raw), "forge_expert_linear_backward")


def _stacked(dev: int, W, m, v, qscales, name: str):
    """Addresses of the experts' weights and states [E, F, D], checked as those of one matrix [E F, D], and their format."""
    flat = [None if t is None else t.view(-1, W.shape[2]) if t.is_contiguous() and t.shape == W.shape else t for t in (W, m, v)]
    _states(dev, flat[0], flat[1], flat[2], qscales)
    return [_take(W, _BF16, tuple(W.shape), dev, name)] + [_fg._ptr(t) for t in (m, v, qscales)], _fg._state_of(m, v)


def expert_linear_backward_step(dY, X, W, offsets, dX=None, m=None, v=None, qscales=None, opt: str = "adamw", hp: Any = None,
                                step: int = 1, seed: int = 0, stream=None) -> None:
    """The same backward pass with the fused step in place of dW: dX (None: not computed) from the weights as they are, and
    W, m, v [E, d_out, d_in] updated in place; qscales as fused_dw_step takes them for one matrix of E d_out rows."""
    dev, R, D, E, F = _grouped(X, W, "W")
    shape = _shape(ExpertLinearShape, R, E, D, F, 0)
    dy, x = _take(dY, _BF16, (R, F), dev, "dY"), _take(X, _BF16, (R, D), dev, "X")
    o, dx = _take(offsets, torch.int32, (E + 1,), dev, "offsets"), _take(dX, _BF16, (R, D), dev, "dX")
    (w, *states), state = _stacked(dev, W, m, v, qscales, "W")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_expert_linear_workspace", dev, stream, raw, 1)
    st = _fg.lib().forge_expert_linear_backward_step(dy, x, w, o, dx, *states, ws, n, state, _fg.OPT_KINDS[opt], _fg._hp_arg(hp),
                                                     shape.arg, int(step), int(seed) & (2**64 - 1), raw)
    _fg._check(st, "forge_expert_linear_backward_step")


def expert_gated_mlp(X, Wg, Wu, Wd, offsets, Y, G=None, U=None, act: str = "silu", stream=None) -> None:
    """gated_mlp with each expert's weights for its rows, as expert_linear: Wg and Wu [E, F, D], Wd [E, D, F]; X and Y
    [R, D]; G and U [R, F], both or neither, for the backward pass."""
    dev, R, D, E, F = _grouped(X, Wg, "Wg")
    shape = _shape(ExpertGatedShape, R, E, D, F, _one_of(ACTIVATIONS, act, "act"), 0)
    args = [_take(t, dt, s, dev, name) for t, dt, s, name in (
        (X, _BF16, (R, D), "X"), (Wg, _BF16, (E, F, D), "Wg"), (Wu, _BF16, (E, F, D), "Wu"), (Wd, _BF16, (E, D, F), "Wd"),
        (offsets, torch.int32, (E + 1,), "offsets"), (Y, _BF16, (R, D), "Y"), (G, _BF16, (R, F), "G"), (U, _BF16, (R, F), "U"))]
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_expert_gated_mlp_workspace", dev, stream, raw, 0)
    _fg._check(_fg.lib().forge_expert_gated_mlp(*args, ws, n, shape.arg, raw), "forge_expert_gated_mlp")


def expert_gated_mlp_backward(dY, X, G, U, Wg, Wu, Wd, offsets, dX, dWg, dWu, dWd, act: str = "silu", stream=None) -> None:
    """The gradients of expert_gated_mlp, bf16, from dY [R, D] and the forward pass's X, G and U.  dX may be None."""
    dev, R, D, E, F = _grouped(X, Wg, "Wg")
    shape = _shape(ExpertGatedShape, R, E, D, F, _one_of(ACTIVATIONS, act, "act"), 0)
    args = [_take(t, dt, s, dev, name) for t, dt, s, name in (
        (dY, _BF16, (R, D), "dY"), (X, _BF16, (R, D), "X"), (G, _BF16, (R, F), "G"), (U, _BF16, (R, F), "U"),
        (Wg, _BF16, (E, F, D), "Wg"), (Wu, _BF16, (E, F, D), "Wu"), (Wd, _BF16, (E, D, F), "Wd"),
        (offsets, torch.int32, (E + 1,), "offsets"), (dX, _BF16, (R, D), "dX"), (dWg, _BF16, (E, F, D), "dWg"),
        (dWu, _BF16, (E, F, D), "dWu"), (dWd, _BF16, (E, D, F), "dWd"))]
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_expert_gated_mlp_workspace", dev, stream, raw, 1)
    _fg._check(_fg.lib().forge_expert_gated_mlp_backward(*args, ws, n, shape.arg, raw), "forge_expert_gated_mlp_backward")


def expert_gated_mlp_backward_step(dY, X, G, U, gate, up, down, offsets, dX=None, act: str = "silu", opt: str = "adamw",
                                   hp: Any = None, step: int = 1, stream=None) -> None:
    """gated_mlp_backward_step with each expert's weights: gate, up and down are (W, m, v, qscales, seed) with W, m, v
    [E, F, D] ([E, D, F] for down) and qscales of one matrix of E F (E D) rows."""
    dev, R, D, E, F = _grouped(X, gate[0], "gate's W")
    shape = _shape(ExpertGatedShape, R, E, D, F, _one_of(ACTIVATIONS, act, "act"), 0)
    args = [_take(t, _BF16, s, dev, name) for t, s, name in (
        (dY, (R, D), "dY"), (X, (R, D), "X"), (G, (R, F), "G"), (U, (R, F), "U"))]
    layers, kinds = [], set()
    for (W, m, v, q, seed), s, name in ((gate, (E, F, D), "gate"), (up, (E, F, D), "up"), (down, (E, D, F), "down")):
        _take(W, _BF16, s, dev, f"{name}'s W")
        ptrs, state = _stacked(dev, W, m, v, q, f"{name}'s W")
        kinds.add(state)
        layers.append(_fg.ForgeLayer(None, None, *ptrs, 0, 0, 0, int(seed) & (2**64 - 1)))
    if len(kinds) > 1:
        raise TypeError("the three layers must use the same state format")
    o, dx = _take(offsets, torch.int32, (E + 1,), dev, "offsets"), _take(dX, _BF16, (R, D), dev, "dX")
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_expert_gated_mlp_workspace", dev, stream, raw, 1)
    st = _fg.lib().forge_expert_gated_mlp_backward_step(
        *args, *(ctypes.byref(a) for a in layers), o, dx, ws, n, kinds.pop(), _fg.OPT_KINDS[opt], _fg._hp_arg(hp), shape.arg,
        int(step), raw)
    _fg._check(st, "forge_expert_gated_mlp_backward_step")


# ------------------------------------------------------------------ dropout


def dropout(x, y, p: float, seed: int = 0, step: int = 0, residual=None, stream=None) -> None:
    """y = dropout(x) (+ residual): each element is 0 with probability p (rounded to 2^-16), else x / (1 - p).  x,
    residual and y bf16 or FP32, of one shape and type.  The mask is made from seed, step and the element's place and is
    never stored.  step: a number, or an int64 tensor of one element on the device, which a captured call reads
    at each replay."""
    dev = _device(x)
    dt, shape = x.dtype, tuple(x.shape)
    at = None
    if torch.is_tensor(step):
        at, step = _take(step.view(-1) if step.dim() == 0 else step, torch.int64, (1,), dev, "step"), 0
    _fg._check(_fg.lib().forge_dropout(
        _take(x, dt, shape, dev, "x"), _take(residual, dt, shape, dev, "residual"), _take(y, dt, shape, dev, "y"), x.numel(),
        _type(x, "x"), float(p), int(seed) & (2**64 - 1), int(step) & (2**64 - 1), at, _raw_stream(stream, dev)), "forge_dropout")


def dropout_backward(dy, dx, p: float, seed: int = 0, step: int = 0, stream=None) -> None:
    """dx of dropout from dy and the forward pass's p, seed and step.  (The gradient of residual is dy.)"""
    dropout(dy, dx, p, seed=seed, step=step, stream=stream)


# ------------------------------------------------------------------ preference loss


def preference_loss(nll, ref, offsets, loss, reward=None, slope=None, mask=None, beta: float = 0.1, kind: str = "sigmoid",
                    smoothing: float = 0.0, margin: float = 0.0, mean: bool = False, stream=None) -> None:
    """loss [P] of P pairs of sequences: nll and ref [T], each token's -log probability under the model (what
    linear_cross_entropy leaves) and under the reference (None: 0); sequence i is tokens offsets[i] .. offsets[i+1]-1
    (int32 [2P+1] on the device), the chosen ones first, then the rejected ones; tokens where mask (bool [T]) is False do
    not count.  score = sum of ref - nll (mean=True: the mean), z = beta (chosen - rejected) - margin; kind "sigmoid"
    (-log sigmoid(z), with label smoothing), "hinge" (max(0, 1 - z)) or "ipo" (((z - 1/2) / beta)^2).  reward [2P] = beta
    score; slope [2P] is what the backward pass needs.  FP32 but for offsets and mask."""
    dev = _device(nll)
    T, P = _vector(nll, "nll"), _vector(loss, "loss")
    shape = _shape(PreferenceShape, T, P, _one_of(PREFERENCES, kind, "kind"), int(bool(mean)), float(beta), float(smoothing),
                   float(margin), 0)
    args = [_take(t, dt, s, dev, name) for t, dt, s, name in (
        (nll, _F32, (T,), "nll"), (ref, _F32, (T,), "ref"), (mask, torch.bool, (T,), "mask"),
        (offsets, torch.int32, (2 * P + 1,), "offsets"), (loss, _F32, (P,), "loss"), (reward, _F32, (2 * P,), "reward"),
        (slope, _F32, (2 * P,), "slope"))]
    raw = _raw_stream(stream, dev)
    ws, n, _hold = _workspace(shape, "forge_preference_loss_workspace", dev, stream, raw)
    _fg._check(_fg.lib().forge_preference_loss(*args, ws, n, shape.arg, raw), "forge_preference_loss")


def preference_loss_backward(dloss, slope, offsets, dnll, mask=None, stream=None) -> None:
    """dnll [T], the gradient of each token's nll (linear_cross_entropy's dloss), from dloss [P] and the forward pass's
    slope [2P]; 0 for tokens that do not count."""
    dev = _device(dnll)
    T, P = _vector(dnll, "dnll"), _vector(dloss, "dloss")
    shape = _shape(PreferenceShape, T, P, 0, 0, 1.0, 0.0, 0.0, 0)
    args = [_take(t, dt, s, dev, name) for t, dt, s, name in (
        (dloss, _F32, (P,), "dloss"), (slope, _F32, (2 * P,), "slope"), (mask, torch.bool, (T,), "mask"),
        (offsets, torch.int32, (2 * P + 1,), "offsets"), (dnll, _F32, (T,), "dnll"))]
    _fg._check(_fg.lib().forge_preference_loss_backward(*args, shape.arg, _raw_stream(stream, dev)),
               "forge_preference_loss_backward")


# ------------------------------------------------------------------ how the products are cut


def _launch_shape(name: str, shape, launch: int) -> dict:
    vals = [ctypes.c_int32() for _ in range(4)]
    _fg._check(getattr(_fg.lib(), name)(shape.arg, launch, *[ctypes.byref(v) for v in vals]), name)
    return dict(zip(("tile_cols", "whole", "cut", "parts"), (v.value for v in vals)))


def gated_launch_shape(T: int, d_model: int, d_ff: int, launch: str) -> dict:
    """Tile columns (0: the few-token kernel), whole and cut tiles and parts of a launch of the gated block: "up" (gate
    and up projection), "down", "dh", "grads" (dX and the weights' gradients)."""
    return _launch_shape("forge_gated_mlp_launch_shape", _shape(GatedShape, T, d_model, d_ff, 0, 0),
                         _one_of({"up": 0, "down": 1, "dh": 2, "grads": 3}, launch, "launch"))


def loss_launch_shape(T: int, vocab: int, d_model: int, launch: str) -> dict:
    """The same of the head's loss: "stats" (forward), "g" and "grads" (dX and dW) of the backward pass's first piece of
    the vocabulary."""
    return _launch_shape("forge_linear_cross_entropy_launch_shape", _shape(LossShape, T, vocab, d_model, -100, 0),
                         _one_of({"stats": 0, "g": 1, "grads": 2}, launch, "launch"))
