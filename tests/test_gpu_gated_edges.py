"""The gated block's derivative far out (needs a GB300)."""
import pytest
import torch

import backward_optimizer_gb300 as fg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
@pytest.mark.parametrize("size", [1e4, 1e13, 3e19, 1e38])
def test_slopes_of_gates_of_any_finite_size(act, size):
    """act'(g) is 1 far above zero and 0 far below, up to the largest numbers: with U = 1, dY = 1 and Wd = I, dG is
    the slope itself, and dWg = dG^T X shows it."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    T, D, F = 2, 8, 8
    b = dict(dtype=torch.bfloat16, device="cuda")
    eye = torch.eye(8, **b)
    G = torch.full((T, F), size, **b)
    G[1] = -size
    X = torch.zeros(T, D, **b)
    X[0, 0], X[1, 1] = 1, 1
    dY, U = torch.ones(T, D, **b), torch.ones(T, F, **b)
    dX, dWg, dWu, dWd = (torch.full(s, float("nan"), **b) for s in ((T, D), (F, D), (F, D), (D, F)))
    fg.gated_mlp_backward(dY, X, G, U, eye, torch.zeros_like(eye), eye, dX, dWg, dWu, dWd, act=act)
    assert fg.sync_status() == 0
    assert (dWg[:, 0] == 1).all() and (dWg[:, 1] == 0).all()
    assert (dX[0] == 1).all() and (dX[1] == 0).all()
