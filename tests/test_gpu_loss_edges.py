"""The head's loss where one token's numbers are not finite (needs a GB300): what the formulas give the others
stays theirs."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import operators_reference as ref
from tests.operators_reference import F64, U8, acc, assert_close, rounded

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _inputs(T, V, D, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=gen, device="cuda") / D ** 0.5).bfloat16()
    t = torch.randint(V, (T,), generator=gen, device="cuda")
    return x, w, t, torch.rand(T, generator=gen, device="cuda") / T


# the first gradient launch finds the largest dloss itself, and a launch of its own does
@pytest.mark.parametrize("T, V, D", [(300, 777, 128), (1500, 777, 128)])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_a_dloss_that_is_not_finite_stays_in_its_row(T, V, D, bad):
    x, w, t, dloss = _inputs(T, V, D, 1)
    dloss[7] = bad
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fg.linear_cross_entropy(x, w, t, loss, lse)
    dX, dW = torch.empty_like(x), torch.empty_like(w)
    fg.linear_cross_entropy_backward(x, w, t, lse, dloss, dX, dW)
    assert fg.sync_status() == 0
    assert not torch.isfinite(dX[7]).any()
    rest = torch.arange(T, device="cuda") != 7
    X, W = x.to(F64), w.to(F64)
    _, wlse, g, logits = ref.loss_and_gradient(X, W, t, torch.where(rest, dloss, 0.0).to(F64), IGNORE)
    # as test_gpu_loss.py derives them: p's error from the logit's and lse's, then g's and dX's roundings
    el = acc(logits, D)
    es = el.max(1).values + (256 + V / 2048) * 2.0 ** -24 + 2.0 ** -21 * (1 + logits.abs().max(1).values)
    eg = (el + es[:, None] + 2.0 ** -20 * (1 + logits.abs())) * torch.where(rest, dloss, 0.0)[:, None] * \
        (logits - wlse[:, None]).exp() + 2.0 ** -22 * g.abs()
    d = g @ W
    tol = (1 + U8) * (rounded(g, W) + acc(d, V) + eg @ W.abs()) + U8 * d.abs() + 1e-30
    assert_close(dX[rest], d[rest], tol[rest], "dX of the other tokens")


@pytest.mark.parametrize("T, V, D", [(40, 300, 64), (3, 5001, 64)])
def test_an_infinite_logit(T, V, D):
    """log sum exp with one term +inf is +inf, and so is the loss of every other target; a row whose logits are
    all -inf has -inf."""
    x, w, t, _ = _inputs(T, V, D, 2)
    w[:, 0] = w[:, 0].abs() + 2 ** -10
    w[5, 0] = -1.0
    x[1, 0] = float("inf")     # +inf everywhere but at entry 5, which is -inf
    x[2, 0] = float("-inf")    # +inf at entry 5 alone, -inf elsewhere
    t[1], t[2] = 5, 7
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fg.linear_cross_entropy(x, w, t, loss, lse)
    assert fg.sync_status() == 0
    want = torch.logsumexp(x.to(F64) @ w.to(F64).T, 1)
    inf = float("inf")
    assert [float(v) for v in want[1:3]] == [inf, inf]
    assert [float(v) for v in lse[1:3]] == [inf, inf] and [float(v) for v in loss[1:3]] == [inf, inf]
    assert torch.isfinite(lse[0]) and torch.isfinite(lse[3:]).all()
