"""Modules around the fused layers: the norm, the gated feed-forward block (dense, or one for each expert), dropout on a
residual branch, the head with its loss, and the preference loss behind it.

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

With experts, dropout and pairs of sequences (rows sorted by expert; head made with reduction="none"):

    h = dropout(experts(norm1(x)[order], offsets)[place], residual=x)
    loss, reward = preference(head(norm2(h), target), ref_nll, sequences)
    loss.mean().backward()
"""
from __future__ import annotations

import collections
from typing import Any, Optional

import torch

from . import operators as ops
from .autograd import _MOMENTS, _STATE_DTYPES, Stepped, once

__all__ = ["ForgeNorm", "ForgeGatedMLP", "ForgeExpertMLP", "ForgeDropout", "ForgeHeadLoss", "ForgePreferenceLoss"]


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


class _ExpertFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, offsets, block, want_dx):
        X = x.detach().contiguous()
        F = block.gate.shape[1]
        Y = torch.zeros_like(X)
        G, U = (torch.empty(X.shape[0], F, dtype=torch.bfloat16, device=X.device) for _ in range(2))
        ops.expert_gated_mlp(X, block.gate.data, block.up.data, block.down.data, offsets, Y, G, U, act=block.act)
        ctx.save_for_backward(X, G, U, offsets)
        ctx.block, ctx.want_dx = block, want_dx
        return Y

    @staticmethod
    @once("ForgeExpertMLP")
    def backward(ctx, grad_out):
        X, G, U, offsets = ctx.saved_tensors
        b = ctx.block
        b._once()
        dX = torch.zeros_like(X) if ctx.want_dx else None
        ops.expert_gated_mlp_backward_step(grad_out.to(torch.bfloat16).contiguous(), X, G, U, b._layer("gate", b.seed),
                                           b._layer("up", b.seed + 1), b._layer("down", b.seed + 2), offsets, dX, act=b.act,
                                           opt=b.opt, hp=b.hp, step=b.step)
        b._done()
        return dX, None, None, None


class ForgeExpertMLP(_Trained):
    """ForgeGatedMLP with a block for each expert: rows offsets[e] .. offsets[e+1]-1 of x [rows, d_model] go through expert e
    (offsets int32 [experts + 1] on the device, never read on the host); rows of no expert give 0.  Every expert takes the
    optimizer step, with a gradient of zero where it had no row.  Arguments as for ForgeGatedMLP; seed, seed + 1 and
    seed + 2 are the three stacked matrices'."""

    def __init__(self, d_model: int, d_ff: int, experts: int, act: str = "silu", opt: str = "adamw", hp: Any = None,
                 state: str = "fp32", seed: int = 0, device=None, init_std: float = 0.02):
        if act not in ops.ACTIVATIONS:
            raise ValueError(f"act: {act!r}, expected one of {list(ops.ACTIVATIONS)}")
        super().__init__({"gate": (experts, d_ff, d_model), "up": (experts, d_ff, d_model), "down": (experts, d_model, d_ff)},
                         opt, hp, state, seed, device, init_std)
        self.act = act

    def forward(self, x: torch.Tensor, offsets: torch.Tensor) -> torch.Tensor:
        if x.dtype != torch.bfloat16:
            raise TypeError("ForgeExpertMLP takes bfloat16 inputs")
        if x.dim() != 2:
            raise ValueError(f"x: {x.dim()} dimensions, expected 2")
        if not torch.is_grad_enabled():
            Y = torch.zeros_like(x, memory_format=torch.contiguous_format)
            ops.expert_gated_mlp(x.contiguous(), self.gate.data, self.up.data, self.down.data, offsets, Y, act=self.act)
            return Y
        want_dx = x.requires_grad
        anchor = x if want_dx else x.detach().requires_grad_(True)
        self._pending = self.step
        return _ExpertFn.apply(anchor, offsets, self, want_dx)

    def extra_repr(self) -> str:
        e, f, d = self.gate.shape
        return f"d_model={d}, d_ff={f}, experts={e}, act={self.act}, opt={self.opt}, step={self.step}"


class _DropoutFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, step):
        X = x.detach().contiguous()
        y = torch.empty_like(X)
        ops.dropout(X, y, p, seed=seed, step=step, residual=None if residual is None else residual.detach().contiguous())
        ctx.p, ctx.seed, ctx.step, ctx.dtype, ctx.has_residual = p, seed, step, x.dtype, residual is not None
        ctx.version = step._version if torch.is_tensor(step) and not step.is_inference() else None
        return y

    @staticmethod
    @once("ForgeDropout")
    def backward(ctx, grad_out):
        dx = None
        if ctx.version is not None and ctx.step._version != ctx.version:
            raise RuntimeError("ForgeDropout: step was changed between the forward and the backward pass")
        if ctx.needs_input_grad[0]:
            dy = grad_out.to(ctx.dtype).contiguous()
            dx = torch.empty_like(dy)
            ops.dropout_backward(dy, dx, ctx.p, seed=ctx.seed, step=ctx.step)
        return dx, grad_out if ctx.has_residual else None, None, None, None


class ForgeDropout(Stepped):
    """dropout(x) (+ residual, of its shape and type), bf16 or FP32, whose mask is made again in the backward pass and never
    stored.  In training mode each forward takes a mask of its own: number `step`, from 1, which goes into the state dict;
    seed is distinct from other dropouts'.  In evaluation mode x (+ residual).

    forward's step: the mask's number instead, and the module's own stays as it is: a number, or an int64 tensor of one
    element on the device that holds its value until the backward pass is through.  A captured forward replays with its
    mask, or with the one that such a tensor says at the replay.

    A forward that a backward pass computes again (torch.utils.checkpoint) takes its mask again.  It is known by a
    number that both draw from PyTorch's CPU generator, which checkpoint sets back; an error is raised where it does not
    (preserve_rng_state=False), where over 1024 forwards lie between, and where forwards that are still to be computed again
    began from the same state of that generator.  Other forwards draw none."""

    _MOST = 1024  # forwards that are known

    def __init__(self, p: float = 0.1, seed: int = 0):
        if not 0.0 <= p <= 1.0:
            raise ValueError(f"p: {p}, expected a number between 0 and 1")
        super().__init__()
        self.p, self.seed = float(p), int(seed)
        # by the number drawn: the forward's step (None: it may be one of several), and whether it has been computed again
        self._masks: collections.OrderedDict = collections.OrderedDict()

    def __setstate__(self, state):
        super().__setstate__(state)
        self.__dict__.setdefault("_masks", collections.OrderedDict())  # pickled before there were any

    def _take_step(self) -> int:
        """The step of a forward that begins here."""
        again = torch._C._current_graph_task_id() >= 0  # a backward pass is running on this thread
        # a forward that is to be computed again runs without gradients, or with hooks on the tensors that it saves (drawing
        # for every one would cost 14 us of the host's time)
        if not again and torch.is_grad_enabled() and torch._C._autograd._top_saved_tensors_default_hooks(True) is None:
            self.step += 1
            return self.step - 1
        drawn = int(torch.empty((), dtype=torch.int64, device="cpu").random_())
        if again:
            step, _ = self._masks.get(drawn, (None, False))
            if step is None:
                raise RuntimeError("ForgeDropout: a backward pass computes a forward again and its mask is not known, since "
                                   "PyTorch's CPU generator was not set back to that forward's state alone; pass step=")
            self._masks[drawn] = step, True
            return step
        step, self.step = self.step, self.step + 1
        _, through = self._masks.pop(drawn, (None, True))
        self._masks[drawn] = step if through else None, False
        if len(self._masks) > self._MOST:
            self._masks.popitem(last=False)
        return step

    def forward(self, x: torch.Tensor, residual: Optional[torch.Tensor] = None, step=None) -> torch.Tensor:
        if x.dtype not in (torch.bfloat16, torch.float32):
            raise TypeError("ForgeDropout takes bfloat16 or FP32 inputs")
        if residual is not None:
            if residual.dtype != x.dtype:
                raise TypeError(f"residual: dtype {residual.dtype}, expected {x.dtype}")
            if residual.shape != x.shape or residual.device != x.device:
                raise ValueError(f"residual: shape {tuple(residual.shape)} on {residual.device}, expected {tuple(x.shape)} on {x.device}")
        if not self.training:
            return x if residual is None else x + residual
        return _DropoutFn.apply(x, residual, self.p, self.seed, self._take_step() if step is None else step)

    def extra_repr(self) -> str:
        return f"p={self.p}, seed={self.seed}, step={self.step}"


class _HeadFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, target, head, want_dx):
        X, t = _rows(x.detach()), target.reshape(-1).contiguous()
        loss, lse = head._losses(X, t)
        share = head._share(t) if head.reduction == "mean" else None
        ctx.save_for_backward(X, t, lse, share)
        ctx.head, ctx.want_dx, ctx.shape = head, want_dx, x.shape
        return loss.view(target.shape) if share is None else (loss * share).sum()

    @staticmethod
    @once("ForgeHeadLoss")
    def backward(ctx, grad_out):
        X, t, lse, share = ctx.saved_tensors
        h = ctx.head
        h._once()
        dX = torch.empty_like(X) if ctx.want_dx else None
        W, m, v, q, seed = h._layer("weight", h.seed)
        dloss = grad_out.float().reshape(-1).contiguous() if share is None else share * grad_out
        ops.linear_cross_entropy_step(X, W, t, lse, dloss, dX, m, v, q, ignore_index=h.ignore_index, opt=h.opt,
                                      hp=h.hp, step=h.step, seed=seed)
        h._done()
        return (None if dX is None else dX.view(ctx.shape)), None, None, None


class ForgeHeadLoss(_Trained):
    """The mean softmax cross entropy of the logits x weight^T over the tokens whose target is not
    ignore_index (0 where there are none), trained by its backward pass; the logits never exist.

    reduction="none": each token's loss instead, in target's shape (0 where it is ignored).
    x [..., d_model] bf16, target [...] int64, weight [vocab, d_model].  opt, hp, state and seed as for
    ForgeLinear (int8 states need d_model to be a multiple of 64)."""

    reduction = "mean"  # of modules pickled before there was a choice

    def __init__(self, d_model: int, vocab: int, opt: str = "adamw", hp: Any = None, state: str = "fp32", seed: int = 0,
                 ignore_index: int = -100, device=None, init_std: float = 0.02, reduction: str = "mean"):
        if reduction not in ("mean", "none"):
            raise ValueError(f"reduction: {reduction!r}, expected 'mean' or 'none'")
        super().__init__({"weight": (vocab, d_model)}, opt, hp, state, seed, device, init_std)
        self.ignore_index, self.reduction = int(ignore_index), reduction

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
            loss = self._losses(_rows(x), t)[0]
            return loss.view(target.shape) if self.reduction == "none" else (loss * self._share(t)).sum()
        want_dx = x.requires_grad
        anchor = x if want_dx else x.detach().requires_grad_(True)
        self._pending = self.step
        return _HeadFn.apply(anchor, target, self, want_dx)

    def extra_repr(self) -> str:
        v, d = self.weight.shape
        return f"d_model={d}, vocab={v}, opt={self.opt}, ignore_index={self.ignore_index}, step={self.step}"


class _PreferenceFn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, nll, ref, offsets, mask, module):
        n = nll.detach().reshape(-1).contiguous()
        P = (offsets.shape[0] - 1) // 2
        loss, reward, slope = (_f32(k, n.device) for k in (P, 2 * P, 2 * P))
        r, m = (None if t is None else t.detach().reshape(-1).contiguous() for t in (ref, mask))
        ops.preference_loss(n, r, offsets, loss, reward, slope, mask=m, **module.options)
        ctx.save_for_backward(slope, offsets, m)
        ctx.shape = nll.shape
        ctx.mark_non_differentiable(reward)
        return loss, reward

    @staticmethod
    @once("ForgePreferenceLoss")
    def backward(ctx, grad_loss, _):
        slope, offsets, mask = ctx.saved_tensors
        dnll = _f32(ctx.shape.numel(), slope.device)
        ops.preference_loss_backward(grad_loss.float().contiguous(), slope, offsets, dnll, mask=mask)
        return dnll.view(ctx.shape), None, None, None, None


class ForgePreferenceLoss(torch.nn.Module):
    """The loss of each of P pairs of sequences, and the reward of each of the 2 P sequences (chosen ones first; not
    differentiable), from each token's -log probability under the model (ForgeHeadLoss with reduction="none") and under the
    reference (None: 0).  offsets int32 [2P + 1] on the device: where the sequences lie among the tokens; mask: tokens that
    count.  beta, kind ("sigmoid", "hinge", "ipo"), smoothing, margin and mean as for operators.preference_loss."""

    def __init__(self, beta: float = 0.1, kind: str = "sigmoid", smoothing: float = 0.0, margin: float = 0.0, mean: bool = False):
        if kind not in ops.PREFERENCES:
            raise ValueError(f"kind: {kind!r}, expected one of {list(ops.PREFERENCES)}")
        super().__init__()
        self.options = dict(beta=float(beta), kind=kind, smoothing=float(smoothing), margin=float(margin), mean=bool(mean))

    def forward(self, nll: torch.Tensor, ref: Optional[torch.Tensor], offsets: torch.Tensor, mask: Optional[torch.Tensor] = None):
        if offsets.dim() != 1 or offsets.shape[0] % 2 == 0:
            raise ValueError(f"offsets: shape {tuple(offsets.shape)}, expected (2 P + 1,)")
        return _PreferenceFn.apply(nll, ref, offsets, mask, self)

    def extra_repr(self) -> str:
        return ", ".join(f"{k}={v}" for k, v in self.options.items())
