"""The operators around the fused layers: the norm, the gated feed-forward block, and the cross
entropy of a linear head, each with its backward pass.

Like the rest of the binding this module checks and marshals arguments; the computation is the
library's.  Results are written to the tensors passed for them.  Tensors are contiguous and on the
current device.  Workspace comes from PyTorch's allocator, on the stream that the call runs on.
`include/forge.h` documents every operator's formulas, types and special cases.
"""
from __future__ import annotations

import ctypes
from typing import Any

import torch

import backward_optimizer_gb300 as _fg

NORM_KINDS = {"layer": 0, "rms": 1}
ACTIVATIONS = {"silu": 0, "gelu_tanh": 1, "relu": 2}
_TYPES = {torch.bfloat16: 0, torch.float32: 1}
_BF16, _F32 = (torch.bfloat16,), (torch.float32,)


class NormShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("D", ctypes.c_int64), ("kind", ctypes.c_int32), ("x_type", ctypes.c_int32),
                ("w_type", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class GatedShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("d_model", ctypes.c_int64), ("d_ff", ctypes.c_int64), ("act", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class LossShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("vocab", ctypes.c_int64), ("d_model", ctypes.c_int64),
                ("ignore_index", ctypes.c_int64), ("reserved", ctypes.c_int64)]


def declare(L: ctypes.CDLL) -> None:
    """Argument types of the library's functions that this module calls."""
    vp, i32, i64, u64, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float
    norm, gated, loss = (ctypes.POINTER(t) for t in (NormShape, GatedShape, LossShape))
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
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, ctypes.c_int
    for name, args in {
        "forge_layer_norm_backward_workspace": [norm],
        "forge_gated_mlp_workspace": [gated, i32],
        "forge_linear_cross_entropy_workspace": [loss, i32],
    }.items():
        f = getattr(L, name)
        f.argtypes, f.restype = args, i64


_bytes: dict = {}  # workspace sizes by device, function and shape: the same for the same sizes


def _workspace(x, stream, name: str, shape, sizes: tuple, *more):
    """A workspace of the size that `name` answers for `shape`, from the memory pool of the stream."""
    key = (x.device.index, name, sizes)
    n = _bytes.get(key)
    if n is None:
        n = getattr(_fg.lib(), name)(ctypes.byref(shape), *more)
        if n < 0:  # the call itself says what is wrong
            return None, 0
        if len(_bytes) >= 4096:
            _bytes.clear()
        _bytes[key] = n
    if n == 0:
        return None, 0
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=x.device), n
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_fg._stream(stream))
    with torch.cuda.stream(s):
        return torch.empty(n, dtype=torch.uint8, device=x.device), n


def _here(x, name: str) -> None:
    if not x.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if x.device.index != torch.cuda.current_device():
        raise ValueError(f"{name}: on {x.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _same_device(*ts) -> None:
    if len({t.device for t in ts if t is not None}) > 1:
        raise ValueError("tensors must live on one device")


def _one_of(table: dict, key: str, name: str) -> int:
    if key not in table:
        raise ValueError(f"{name}: {key!r}, expected one of {list(table)}")
    return table[key]


def _matrix(t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: {t.dim()} dimensions, expected 2")
    return t.shape


# ------------------------------------------------------------------ norm


def _norm_shape(x, weight, kind: str) -> NormShape:
    T, D = _matrix(x, "x")
    for t, name in ((x, "x"), (weight, "weight")):
        if t.dtype not in _TYPES:
            raise TypeError(f"{name}: dtype {t.dtype}, expected one of {[str(d) for d in _TYPES]}")
    return NormShape(T, D, _one_of(NORM_KINDS, kind, "kind"), _TYPES[x.dtype], _TYPES[weight.dtype], 0)


def layer_norm(x, weight, bias, y, mean=None, rstd=None, eps: float = 1e-5, kind: str = "layer", stream=None) -> None:
    """y [T, D] = norm(x) * weight (+ bias) row by row: the layer norm, or with kind="rms" the RMS norm
    (no mean, no bias).  x and y bf16 or FP32, weight and bias [D] bf16 or FP32.  mean and rstd, FP32 [T],
    are what layer_norm_backward needs."""
    shape = _norm_shape(x, weight, kind)
    T, D = x.shape
    _here(x, "x")
    _same_device(x, weight, bias, y, mean, rstd)
    _fg._expect(weight, (weight.dtype,), (D,), "weight")
    _fg._expect(bias, (weight.dtype,), (D,), "bias")
    _fg._expect(y, (x.dtype,), (T, D), "y")
    _fg._expect(mean, _F32, (T,), "mean")
    _fg._expect(rstd, _F32, (T,), "rstd")
    p = _fg._ptr
    _fg._check(_fg.lib().forge_layer_norm(p(x), p(weight), p(bias), p(y), p(mean), p(rstd), eps, ctypes.byref(shape),
                                          _fg._stream(stream)), "forge_layer_norm")


def layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias=None, add=None, kind: str = "layer",
                        stream=None) -> None:
    """dx [T, D], dweight and dbias (FP32 [D]) of layer_norm from its x and its mean and rstd (RMS norm:
    mean and dbias None).  add [T, D], the gradient along a residual branch past the norm, is added to dx."""
    shape = _norm_shape(x, weight, kind)
    T, D = x.shape
    _here(x, "x")
    _same_device(x, dy, weight, mean, rstd, dx, dweight, dbias, add)
    _fg._expect(weight, (weight.dtype,), (D,), "weight")
    for t, name in ((dy, "dy"), (dx, "dx"), (add, "add")):
        _fg._expect(t, (x.dtype,), (T, D), name)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        _fg._expect(t, _F32, (T,), name)
    for t, name in ((dweight, "dweight"), (dbias, "dbias")):
        _fg._expect(t, _F32, (D,), name)
    p = _fg._ptr
    ws, n = _workspace(x, stream, "forge_layer_norm_backward_workspace", shape,
                       (T, D, shape.kind, shape.x_type, shape.w_type))
    _fg._check(_fg.lib().forge_layer_norm_backward(p(dy), p(x), p(weight), p(mean), p(rstd), p(add), p(dx), p(dweight),
                                                   p(dbias), p(ws), n, ctypes.byref(shape), _fg._stream(stream)),
               "forge_layer_norm_backward")


# ------------------------------------------------------------------ gated feed-forward block


def _gated(X, Wg, Wu, Wd, act: str):
    T, D = _matrix(X, "X")
    F = _matrix(Wg, "Wg")[0]
    _here(X, "X")
    for t, name, shp in ((X, "X", (T, D)), (Wg, "Wg", (F, D)), (Wu, "Wu", (F, D)), (Wd, "Wd", (D, F))):
        _fg._expect(t, _BF16, shp, name)
    return T, D, F, GatedShape(T, D, F, _one_of(ACTIVATIONS, act, "act"), 0)


def gated_mlp(X, Wg, Wu, Wd, Y, G=None, U=None, residual=None, act: str = "silu", stream=None) -> None:
    """Y [T, D] = (act(X Wg^T) * (X Wu^T)) Wd^T (+ residual), everything bf16: X [T, D], Wg and Wu [F, D],
    Wd [D, F].  G and U [T, F], both or neither: X Wg^T and X Wu^T, which the backward pass needs."""
    T, D, F, shape = _gated(X, Wg, Wu, Wd, act)
    for t, name, shp in ((Y, "Y", (T, D)), (residual, "residual", (T, D)), (G, "G", (T, F)), (U, "U", (T, F))):
        _fg._expect(t, _BF16, shp, name)
    _same_device(X, Wg, Wu, Wd, Y, G, U, residual)
    p = _fg._ptr
    ws, n = _workspace(X, stream, "forge_gated_mlp_workspace", shape, (T, D, F, 0), 0)
    _fg._check(_fg.lib().forge_gated_mlp(p(X), p(Wg), p(Wu), p(Wd), p(residual), p(Y), p(G), p(U), p(ws), n,
                                         ctypes.byref(shape), _fg._stream(stream)), "forge_gated_mlp")


def gated_mlp_backward(dY, X, G, U, Wg, Wu, Wd, dX, dWg, dWu, dWd, act: str = "silu", stream=None) -> None:
    """The block's gradients, bf16, from dY [T, D] and the forward pass's X, G and U.  dX may be None."""
    T, D, F, shape = _gated(X, Wg, Wu, Wd, act)
    for t, name, shp in ((dY, "dY", (T, D)), (G, "G", (T, F)), (U, "U", (T, F)), (dX, "dX", (T, D)),
                         (dWg, "dWg", (F, D)), (dWu, "dWu", (F, D)), (dWd, "dWd", (D, F))):
        _fg._expect(t, _BF16, shp, name)
    _same_device(X, dY, G, U, Wg, Wu, Wd, dX, dWg, dWu, dWd)
    p = _fg._ptr
    ws, n = _workspace(X, stream, "forge_gated_mlp_workspace", shape, (T, D, F, 1), 1)
    _fg._check(_fg.lib().forge_gated_mlp_backward(p(dY), p(X), p(G), p(U), p(Wg), p(Wu), p(Wd), p(dX), p(dWg), p(dWu),
                                                  p(dWd), p(ws), n, ctypes.byref(shape), _fg._stream(stream)),
               "forge_gated_mlp_backward")


def gated_mlp_backward_step(dY, X, G, U, gate, up, down, dX=None, act: str = "silu", opt: str = "adamw", hp: Any = None,
                            step: int = 1, stream=None) -> None:
    """The block's backward pass with the fused step: dX (None: not computed) from the weights as they are,
    then W, m, v of the three layers updated in place.  gate, up and down are (W, m, v, qscales, seed), as
    fused_dw_step takes them, all with the same state format."""
    Wg, Wu, Wd = gate[0], up[0], down[0]
    T, D, F, shape = _gated(X, Wg, Wu, Wd, act)
    for t, name, shp in ((dY, "dY", (T, D)), (G, "G", (T, F)), (U, "U", (T, F)), (dX, "dX", (T, D))):
        _fg._expect(t, _BF16, shp, name)
    _same_device(X, dY, G, U, dX, *gate[:4], *up[:4], *down[:4])
    p = _fg._ptr
    arg, states = [], set()
    for W, m, v, q, seed in (gate, up, down):
        _fg._state_args(W, m, v, q)
        states.add(_fg._state_of(m, v))
        arg.append(_fg.ForgeLayer(None, None, p(W), p(m), p(v), p(q), 0, 0, 0, int(seed) & (2**64 - 1)))
    if len(states) > 1:
        raise TypeError("the three layers must use the same state format")
    ws, n = _workspace(X, stream, "forge_gated_mlp_workspace", shape, (T, D, F, 1), 1)
    _fg._check(_fg.lib().forge_gated_mlp_backward_step(
        p(dY), p(X), p(G), p(U), *(ctypes.byref(a) for a in arg), p(dX), p(ws), n, states.pop(), _fg.OPT_KINDS[opt],
        _fg._hp_arg(hp), ctypes.byref(shape), int(step), _fg._stream(stream)), "forge_gated_mlp_backward_step")


# ------------------------------------------------------------------ cross entropy of a linear head


def _loss(X, W, target, ignore_index: int):
    T, D = _matrix(X, "X")
    V = _matrix(W, "W")[0]
    _here(X, "X")
    _fg._expect(X, _BF16, (T, D), "X")
    _fg._expect(W, _BF16, (V, D), "W")
    _fg._expect(target, (torch.int64,), (T,), "target")
    return T, V, D, LossShape(T, V, D, int(ignore_index), 0)


def linear_cross_entropy(X, W, target, loss, lse, ignore_index: int = -100, stream=None) -> None:
    """loss [T] = lse - logit of the target, lse [T] = log sum exp of the logits X W^T (both FP32), without
    the logits in memory: X [T, D] and W [V, D] bf16, target [T] int64.  The loss is 0 where the target is
    ignore_index, NaN at any other target outside 0 .. V-1."""
    T, V, D, shape = _loss(X, W, target, ignore_index)
    _fg._expect(loss, _F32, (T,), "loss")
    _fg._expect(lse, _F32, (T,), "lse")
    _same_device(X, W, target, loss, lse)
    p = _fg._ptr
    ws, n = _workspace(X, stream, "forge_linear_cross_entropy_workspace", shape, (T, V, D, 0), 0)
    _fg._check(_fg.lib().forge_linear_cross_entropy(p(X), p(W), p(target), p(loss), p(lse), p(ws), n,
                                                    ctypes.byref(shape), _fg._stream(stream)),
               "forge_linear_cross_entropy")


def linear_cross_entropy_backward(X, W, target, lse, dloss, dX, dW, ignore_index: int = -100, stream=None) -> None:
    """dX [T, D] and dW [V, D] (bf16, either may be None) given dloss [T], the gradient of each token's loss,
    and the forward pass's lse."""
    T, V, D, shape = _loss(X, W, target, ignore_index)
    for t, name in ((lse, "lse"), (dloss, "dloss")):
        _fg._expect(t, _F32, (T,), name)
    _fg._expect(dX, _BF16, (T, D), "dX")
    _fg._expect(dW, _BF16, (V, D), "dW")
    _same_device(X, W, target, lse, dloss, dX, dW)
    p = _fg._ptr
    ws, n = _workspace(X, stream, "forge_linear_cross_entropy_workspace", shape, (T, V, D, 1), 1)
    _fg._check(_fg.lib().forge_linear_cross_entropy_backward(p(X), p(W), p(target), p(lse), p(dloss), p(dX), p(dW),
                                                             p(ws), n, ctypes.byref(shape), _fg._stream(stream)),
               "forge_linear_cross_entropy_backward")


def linear_cross_entropy_step(X, W, target, lse, dloss, dX=None, m=None, v=None, qscales=None, ignore_index: int = -100,
                              opt: str = "adamw", hp: Any = None, step: int = 1, seed: int = 0, stream=None) -> None:
    """The same backward pass with the fused step in place of dW: dX (None: not computed) from the weights as
    they are, and W, m, v updated in place, as fused_dw_step takes them."""
    T, V, D, shape = _loss(X, W, target, ignore_index)
    for t, name in ((lse, "lse"), (dloss, "dloss")):
        _fg._expect(t, _F32, (T,), name)
    _fg._expect(dX, _BF16, (T, D), "dX")
    _fg._state_args(W, m, v, qscales)
    _same_device(X, W, target, lse, dloss, dX, m, v, qscales)
    p = _fg._ptr
    ws, n = _workspace(X, stream, "forge_linear_cross_entropy_workspace", shape, (T, V, D, 1), 1)
    _fg._check(_fg.lib().forge_linear_cross_entropy_step(
        p(X), p(W), p(target), p(lse), p(dloss), p(dX), p(m), p(v), p(qscales), p(ws), n, _fg._state_of(m, v),
        _fg.OPT_KINDS[opt], _fg._hp_arg(hp), ctypes.byref(shape), int(step), int(seed) & (2**64 - 1),
        _fg._stream(stream)), "forge_linear_cross_entropy_step")
