"""Modules around the fused layers: the norm, the gated feed-forward block, and the head with its loss.

They put the library's operators (operators.py) behind PyTorch autograd, next to `ForgeLinear`
(autograd.py).  The matrices of `ForgeGatedMLP` and `ForgeHeadLoss` are trained as `ForgeLinear`'s is
("FORGE: Fused On-Register Gradient Elimination for Memory-Efficient LLM Training", §2 Methodology, Core
mechanism): the backward pass itself updates them and their optimizer state, their gradients never
exist, and the same limits hold: one backward per forward, no weight shared with another layer of
the same backward, one optimizer step per micro-batch.  `ForgeNorm`'s weight and bias are vectors with
ordinary gradients, for an ordinary optimizer.  No gradient of these modules can be differentiated again:
it raises an error.

    norm1, mlp = ForgeNorm(1024), ForgeGatedMLP(1024, 4096, opt="adamw", hp=hp)
    norm2, head = ForgeNorm(1024), ForgeHeadLoss(1024, vocab, opt="adamw", hp=hp, seed=3)
    h = mlp(norm1(x), residual=x)
    head(norm2(h), target).backward()
"""
from __future__ import annotations

from typing import Any, Optional

import torch

from . import operators as ops
from .autograd import _MOMENTS, _STATE_DTYPES, Stepped, once

__all__ = ["ForgeNorm", "ForgeGatedMLP", "ForgeHeadLoss"]


def _rows(t: torch.Tensor) -> torch.Tensor:
    return t.reshape(-1, t.shape[-1]).contiguous()


def _f32(n: int, device) -> torch.Tensor:
    """FP32 whatever PyTorch's default type is."""
    return torch.empty(n, dtype=torch.float32, device=device)


class _NormFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, kind, eps):
        X = _rows(x.detach())
        y = torch.empty_like(X)
        mean = _f32(X.shape[0], X.device) if kind == "layer" else None
        rstd = _f32(X.shape[0], X.device)
        ops.layer_norm(X, weight, bias, y, mean, rstd, eps=eps, kind=kind)
        ctx.save_for_backward(X, weight, mean, rstd)
        ctx.kind, ctx.has_bias = kind, bias is not None
        return y.view(x.shape)

    @staticmethod
    @once("ForgeNorm")
    def backward(ctx, grad_out):
        X, weight, mean, rstd = ctx.saved_tensors
        dy = _rows(grad_out).to(X.dtype)
        dx, dw = torch.empty_like(X), _f32(X.shape[1], X.device)
        db = torch.empty_like(dw) if ctx.kind == "layer" else None
        ops.layer_norm_backward(dy, X, weight, mean, rstd, dx, dw, db, kind=ctx.kind)
        return (dx.view(grad_out.shape), dw.to(weight.dtype), db.to(weight.dtype) if ctx.has_bias else None, None, None)


class ForgeNorm(torch.nn.Module):
    """Layer norm (kind="layer", with a bias unless bias=False) or RMS norm (kind="rms") over the last
    dimension; inputs bf16 or FP32, weight and bias FP32."""

    def __init__(self, width: int, kind: str = "layer", eps: float = 1e-5, bias: bool = True, device=None):
        super().__init__()
        if kind not in ops.NORM_KINDS:
            raise ValueError(f"kind: {kind!r}, expected one of {list(ops.NORM_KINDS)}")
        dev = torch.device("cuda") if device is None else torch.device(device)
        self.weight = torch.nn.Parameter(torch.ones(width, dtype=torch.float32, device=dev))
        self.bias = (torch.nn.Parameter(torch.zeros(width, dtype=torch.float32, device=dev)) if kind == "layer" and bias
                     else None)
        self.kind, self.eps = kind, float(eps)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        return _NormFn.apply(x, self.weight, self.bias, self.kind, self.eps)

    def extra_repr(self) -> str:
        return f"{self.weight.shape[0]}, kind={self.kind}, eps={self.eps}, bias={self.bias is not None}"


class _Trained(Stepped):
    """Matrices with the optimizer state that their backward pass updates."""

    def __init__(self, shapes: dict, opt: str, hp: Any, state: str, seed: int, device, init_std: float):
        super().__init__()
        if opt not in _MOMENTS:
            raise ValueError(f"unknown optimizer {opt!r}")
        if state not in _STATE_DTYPES:
            raise ValueError("state: 'fp32', 'bf16' or 'int8'")
        dev = torch.device("cuda") if device is None else torch.device(device)
        use_m, use_v = _MOMENTS[opt]
        sdt = _STATE_DTYPES[state]
        for name, shape in shapes.items():
            w = (torch.randn(shape, dtype=torch.float32, device=dev) * init_std).to(torch.bfloat16)
            # the backward itself updates the weight: autograd gives it no gradient
            self.register_parameter(name, torch.nn.Parameter(w, requires_grad=False))
            self.register_buffer(f"{name}_m", torch.zeros(shape, dtype=sdt, device=dev) if use_m else None)
            self.register_buffer(f"{name}_v", torch.zeros(shape, dtype=sdt, device=dev) if use_v else None)
            q = state == "int8" and (use_m or use_v)
            # all-zero codes decode to zero whatever their scale
            self.register_buffer(f"{name}_q", torch.zeros(2 * w.numel() // 64, dtype=torch.float32, device=dev) if q else None)
        self.opt, self.hp, self.seed = opt, hp, int(seed)

    def _layer(self, name: str, seed: int):
        return (getattr(self, name).data, getattr(self, f"{name}_m"), getattr(self, f"{name}_v"),
                getattr(self, f"{name}_q"), seed)

    def _once(self) -> None:
        if self._pending != self.step:
            raise RuntimeError(f"{type(self).__name__}: one backward per forward (the weights were already updated)")

    def _done(self) -> None:
        self._pending = None
        self.step += 1


class _GatedFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, block, want_dx):
        X, R = _rows(x.detach()), None if residual is None else _rows(residual.detach())
        F = block.gate.shape[0]
        Y = torch.empty_like(X)
        G, U = (torch.empty(X.shape[0], F, dtype=torch.bfloat16, device=X.device) for _ in range(2))
        ops.gated_mlp(X, block.gate.data, block.up.data, block.down.data, Y, G, U, residual=R, act=block.act)
        ctx.save_for_backward(X, G, U)
        ctx.block, ctx.want_dx, ctx.has_residual = block, want_dx, residual is not None
        return Y.view(x.shape)

    @staticmethod
    @once("ForgeGatedMLP")
    def backward(ctx, grad_out):
        X, G, U = ctx.saved_tensors
        b = ctx.block
        b._once()
        dY = _rows(grad_out).to(torch.bfloat16)
        dX = torch.empty_like(X) if ctx.want_dx else None
        ops.gated_mlp_backward_step(dY, X, G, U, b._layer("gate", b.seed), b._layer("up", b.seed + 1),
                                    b._layer("down", b.seed + 2), dX, act=b.act, opt=b.opt, hp=b.hp, step=b.step)
        b._done()
        return (None if dX is None else dX.view(grad_out.shape), grad_out if ctx.has_residual else None, None, None)


class ForgeGatedMLP(_Trained):
    """y = (act(x gate^T) * (x up^T)) down^T (+ residual), bf16, trained by its backward pass.

    act: "silu", "gelu_tanh" or "relu".  opt, hp and state as for ForgeLinear (int8 states need d_model
    and d_ff to be multiples of 64).  seed, seed + 1 and seed + 2 are the three matrices'
    stochastic-rounding seeds, distinct from other layers'."""

    def __init__(self, d_model: int, d_ff: int, act: str = "silu", opt: str = "adamw", hp: Any = None,
                 state: str = "fp32", seed: int = 0, device=None, init_std: float = 0.02):
        if act not in ops.ACTIVATIONS:
            raise ValueError(f"act: {act!r}, expected one of {list(ops.ACTIVATIONS)}")
        super().__init__({"gate": (d_ff, d_model), "up": (d_ff, d_model), "down": (d_model, d_ff)}, opt, hp, state, seed,
                         device, init_std)
        self.act = act

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None) -> torch.Tensor:
        for t in (x, residual):
            if t is not None and t.dtype != torch.bfloat16:
                raise TypeError("ForgeGatedMLP takes bfloat16 inputs")
        if not torch.is_grad_enabled():
            X, Y = _rows(x), torch.empty(x.shape, dtype=x.dtype, device=x.device)
            ops.gated_mlp(X, self.gate.data, self.up.data, self.down.data, Y.view(X.shape),
                          residual=None if residual is None else _rows(residual), act=self.act)
            return Y
        want_dx = x.requires_grad
        # autograd calls a backward only for outputs that depend on a tensor requiring grad
        anchor = x if want_dx else x.detach().requires_grad_(True)
        self._pending = self.step
        return _GatedFn.apply(anchor, residual, self, want_dx)

    def extra_repr(self) -> str:
        f, d = self.gate.shape
        return f"d_model={d}, d_ff={f}, act={self.act}, opt={self.opt}, step={self.step}"


class _HeadFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, target, head, want_dx):
        X, t = _rows(x.detach()), target.reshape(-1).contiguous()
        loss, lse = head._losses(X, t)
        share = head._share(t)
        ctx.save_for_backward(X, t, lse, share)
        ctx.head, ctx.want_dx, ctx.shape = head, want_dx, x.shape
        return (loss * share).sum()

    @staticmethod
    @once("ForgeHeadLoss")
    def backward(ctx, grad_out):
        X, t, lse, share = ctx.saved_tensors
        h = ctx.head
        h._once()
        dX = torch.empty_like(X) if ctx.want_dx else None
        W, m, v, q, seed = h._layer("weight", h.seed)
        ops.linear_cross_entropy_step(X, W, t, lse, share * grad_out, dX, m, v, q, ignore_index=h.ignore_index, opt=h.opt,
                                      hp=h.hp, step=h.step, seed=seed)
        h._done()
        return (None if dX is None else dX.view(ctx.shape)), None, None, None


class ForgeHeadLoss(_Trained):
    """The mean softmax cross entropy of the logits x weight^T over the tokens whose target is not
    ignore_index (0 where there are none), trained by its backward pass; the logits never exist.

    x [..., d_model] bf16, target [...] int64, weight [vocab, d_model].  opt, hp, state and seed as for
    ForgeLinear (int8 states need d_model to be a multiple of 64)."""

    def __init__(self, d_model: int, vocab: int, opt: str = "adamw", hp: Any = None, state: str = "fp32", seed: int = 0,
                 ignore_index: int = -100, device=None, init_std: float = 0.02):
        super().__init__({"weight": (vocab, d_model)}, opt, hp, state, seed, device, init_std)
        self.ignore_index = int(ignore_index)

    def _losses(self, X, t):
        loss, lse = (_f32(X.shape[0], X.device) for _ in range(2))
        ops.linear_cross_entropy(X, self.weight.data, t, loss, lse, ignore_index=self.ignore_index)
        return loss, lse

    def _share(self, t):
        """What each token's loss counts for in the mean."""
        counts = t != self.ignore_index
        return counts.float() / counts.sum().clamp_min(1)

    def forward(self, x: torch.Tensor, target: torch.Tensor) -> torch.Tensor:
        if x.dtype != torch.bfloat16:
            raise TypeError("ForgeHeadLoss takes bfloat16 inputs")
        if x.shape[:-1] != target.shape:
            raise ValueError(f"target: shape {tuple(target.shape)}, expected {tuple(x.shape[:-1])}")
        if not torch.is_grad_enabled():
            t = target.reshape(-1).contiguous()
            return (self._losses(_rows(x), t)[0] * self._share(t)).sum()
        want_dx = x.requires_grad
        anchor = x if want_dx else x.detach().requires_grad_(True)
        self._pending = self.step
        return _HeadFn.apply(anchor, target, self, want_dx)

    def extra_repr(self) -> str:
        v, d = self.weight.shape
        return f"d_model={d}, vocab={v}, opt={self.opt}, ignore_index={self.ignore_index}, step={self.step}"
