"""The operators around the fused layers in binary64, and how far the library may be from them.

Plain torch operations on float64 tensors, written from the formulas; nothing of the library.  The
tolerances follow from what the library states it does and were set before it first ran:
- U8: one rounding to bfloat16 (8 significant bits) is off by at most 2^-8 of the value.
- acc(K): the tensor core's FP32 sum over K products, as the parity tests of the weight gradient take
  it: 0.75 (K / 16) 2^-23 of max(|sum|, rms of the sums), at least 2^-20.
- rounded(a, b): a sum of products whose left factors were each rounded to bfloat16: independent
  errors of at most 2^-8 |a b| (standard deviation below 2^-8 / sqrt 3), so 4 * 2^-8 sqrt(sum (a b)^2)
  is about seven standard deviations.
"""
import math

import torch

U8 = 2.0 ** -8
F64 = torch.float64


def acc(c: torch.Tensor, K: int) -> torch.Tensor:
    rms = c.square().mean().sqrt() if c.numel() else torch.zeros((), dtype=F64, device=c.device)
    return max(2.0 ** -20, 0.75 * math.ceil(K / 16) * 2.0 ** -23) * torch.maximum(c.abs(), rms)


def rounded(a: torch.Tensor, b: torch.Tensor) -> torch.Tensor:
    return 4 * U8 * (a.square() @ b.square()).sqrt()


def assert_close(got: torch.Tensor, want: torch.Tensor, tol, what: str) -> None:
    """|got - want| <= tol element by element; NaN and infinities in the same places."""
    got = got.to(F64)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine), f"{what}: not finite in other places"
    over = ((got - want).abs() - tol)[fine] if torch.is_tensor(tol) else ((got - want).abs()[fine] - tol)
    assert over.numel() == 0 or over.max().item() <= 0, (
        f"{what}: {int((over > 0).sum())} of {over.numel()} values out of tolerance, worst by {over.max().item():.3g}")


def act_both(g: torch.Tensor, act: str):
    """act(g) and its derivative."""
    if act == "relu":
        return g.clamp_min(0), (g > 0).to(g.dtype)
    if act == "silu":
        p = torch.sigmoid(g)
        return g * p, p + g * p * (1 - p)
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def norm(x, w, b, eps, kind):
    mean = x.mean(1, keepdim=True) if kind == "layer" else torch.zeros_like(x[:, :1])
    rstd = 1 / ((x - mean).square().mean(1, keepdim=True) + eps).sqrt()
    y = (x - mean) * rstd * w
    return (y if b is None else y + b), mean, rstd


def norm_backward(dy, x, w, mean, rstd, kind):
    xh = (x - mean) * rstd
    g = dy * w
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - g.mean(1, keepdim=True)
    return dx * rstd, (dy * xh).sum(0), dy.sum(0)


def loss_and_gradient(x, w, target, dloss, ignore):
    """loss [T], lse [T], g [T, V] (the gradient with respect to the logits), logits."""
    logits = x @ w.T
    lse = torch.logsumexp(logits, 1)
    counts = target != ignore
    at = torch.where(counts, target, 0)
    loss = torch.where(counts, lse - logits.gather(1, at[:, None])[:, 0], 0.0)
    g = (logits - lse[:, None]).exp()
    g[torch.arange(len(at), device=x.device), at] -= 1
    return loss, lse, g * torch.where(counts, dloss, 0.0)[:, None], logits
