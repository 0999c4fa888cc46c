"""Bounded waits of the products grouped by expert: one that runs out is reported, and the calls behind it are right."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests.test_gpu_waits import _check, _gpu, _rand  # noqa: F401  (the fixture sets a short limit)

pytestmark = pytest.mark.gpu


# row tiles of 32, 64, 128 and 256 rows; a last wave cut along the reduction; gradients on single CTAs and on pairs
@pytest.mark.parametrize("sizes, D, F", [([1, 0, 1], 2048, 1024), ([9, 30, 0, 20], 512, 264), ([70, 0, 50], 256, 512),
                                         ([300, 0, 500], 1024, 1536), ([20, 0, 4, 33] * 20, 512, 512),
                                         ([150, 0, 200], 104, 5000), ([12000, 0, 70], 72, 136)])
def test_experts(sizes, D, F):
    R, E = sum(sizes), len(sizes)
    off = torch.tensor([0] + sizes).cumsum(0).to(torch.int32).cuda()
    X, dY, W = _rand(0, R, D), _rand(1, R, F), _rand(2, E, F, D)
    Y, dX, dW = torch.empty(R, F, dtype=X.dtype, device="cuda"), torch.empty_like(X), torch.empty_like(W)
    _check(lambda: fg.expert_linear(X, W, off, Y), [Y])
    _check(lambda: fg.expert_linear_backward(dY, X, W, off, dX, None), [dX])
    _check(lambda: fg.expert_linear_backward(dY, X, W, off, None, dW), [dW])
    Wu, Wd, G, U = _rand(3, E, F, D), _rand(4, E, D, F), _rand(5, R, F), _rand(6, R, F)
    Z, dZ = torch.empty_like(X), _rand(7, R, D)
    _check(lambda: fg.expert_gated_mlp(X, W, Wu, Wd, off, Z), [Z])
    grads = [torch.empty_like(X), torch.empty_like(W), torch.empty_like(W), torch.empty_like(Wd)]
    _check(lambda: fg.expert_gated_mlp_backward(dZ, X, G, U, W, Wu, Wd, off, *grads), grads)
    w = W.clone()
    m, v = torch.zeros(E, F, D, device="cuda"), torch.zeros(E, F, D, device="cuda")

    def step():
        w.copy_(W)
        m.zero_()
        v.zero_()
        fg.expert_linear_backward_step(dY, X, w, off, None, m, v, opt="adamw", step=1)
    _check(step, [w, m, v])
