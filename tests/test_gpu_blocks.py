"""The modules of blocks.py on the GPU: they make the operators' calls, gradients reach what lies before
them, and a model of them learns."""
import importlib.util
import os

import pytest
import torch

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.blocks import ForgeGatedMLP, ForgeHeadLoss, ForgeNorm
from workloads import Hparams

pytestmark = pytest.mark.gpu

HP = Hparams(lr=1e-2, weight_decay=0.0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _x(*shape, seed=0, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).bfloat16().cuda()


def _same(a, b):
    return (a is None) == (b is None) and (a is None or torch.equal(a, b))


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm(kind):
    n = ForgeNorm(96, kind=kind)
    n.weight.data.copy_(1 + 0.1 * torch.randn(96))
    x = _x(2, 20, 96).requires_grad_(True)
    dy = _x(2, 20, 96, seed=1)
    n(x).backward(dy)
    X, y = x.detach().view(40, 96), torch.empty(40, 96, dtype=torch.bfloat16, device="cuda")
    mean = torch.empty(40, device="cuda") if kind == "layer" else None
    rstd, dx, dw = torch.empty(40, device="cuda"), torch.empty_like(X), torch.empty(96, device="cuda")
    db = torch.empty(96, device="cuda") if kind == "layer" else None
    fg.layer_norm(X, n.weight.data, None if n.bias is None else n.bias.data, y, mean, rstd, kind=kind)
    fg.layer_norm_backward(dy.view(40, 96), X, n.weight.data, mean, rstd, dx, dw, db, kind=kind)
    torch.cuda.synchronize()
    with torch.no_grad():
        assert torch.equal(n(x).view(40, 96), y)
    assert torch.equal(x.grad.view(40, 96), dx) and torch.equal(n.weight.grad, dw)
    assert _same(None if n.bias is None else n.bias.grad, db)


@pytest.mark.parametrize("opt, state", [("adamw", "fp32"), ("lion", "bf16"), ("adamw", "int8"), ("sgd", "fp32")])
def test_gated_mlp(opt, state):
    block = ForgeGatedMLP(128, 320, act="gelu_tanh", opt=opt, hp=HP, state=state, seed=5)
    for step in (1, 2):
        x, r = _x(2, 33, 128, seed=step).requires_grad_(True), _x(2, 33, 128, seed=10).requires_grad_(True)
        dy = _x(2, 33, 128, seed=20 + step, std=0.1)
        layers = [tuple(None if t is None else t.clone() for t in block._layer(n, 0)[:4]) + (5 + i,)
                  for i, n in enumerate(("gate", "up", "down"))]
        y = block(x, residual=r)
        y.backward(dy)
        X, Y, dX = x.detach().view(66, 128), torch.empty(66, 128, dtype=torch.bfloat16, device="cuda"), torch.empty_like(_x(66, 128))
        G, U = (torch.empty(66, 320, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        fg.gated_mlp(X, layers[0][0], layers[1][0], layers[2][0], Y, G, U, residual=r.detach().view(66, 128), act="gelu_tanh")
        fg.gated_mlp_backward_step(dy.view(66, 128), X, G, U, *layers, dX, act="gelu_tanh", opt=opt, hp=HP, step=step)
        assert fg.sync_status() == 0
        assert torch.equal(y.detach().view(66, 128), Y) and torch.equal(x.grad.view(66, 128), dX) and torch.equal(r.grad, dy)
        for want, name in zip(layers, ("gate", "up", "down")):
            assert all(_same(a, b) for a, b in zip(block._layer(name, 0)[:4], want[:4])), name
            assert getattr(block, name).grad is None
        assert block.step == step + 1
    with torch.no_grad():
        Y2 = torch.empty_like(Y)  # the weights as they are now, nothing kept for a backward pass
        fg.gated_mlp(X, block.gate.data, block.up.data, block.down.data, Y2, act="gelu_tanh")
        assert torch.equal(block(x).view(66, 128), Y2)
    with pytest.raises(RuntimeError, match="one backward per forward"):
        y = block(x)
        y.sum().backward(retain_graph=True)
        y.sum().backward()


@pytest.mark.parametrize("state", ["fp32", "bf16", "int8"])
def test_head_loss(state):
    head = ForgeHeadLoss(128, 777, hp=HP, state=state, seed=4)
    x = _x(3, 30, 128).requires_grad_(True)
    t = torch.randint(777, (3, 30), generator=torch.Generator().manual_seed(2)).cuda()
    t[0, :7] = -100
    W, m, v, q, _ = (None if a is None else a if isinstance(a, int) else a.clone() for a in head._layer("weight", 0))
    loss = head(x, t)
    (2 * loss).backward()
    X, tt = x.detach().view(90, 128), t.view(90)
    losses, lse, dX = torch.empty(90, device="cuda"), torch.empty(90, device="cuda"), torch.empty_like(X)
    fg.linear_cross_entropy(X, W, tt, losses, lse)
    share = (tt != -100) / (tt != -100).sum()
    fg.linear_cross_entropy_step(X, W, tt, lse, share * 2, dX, m, v, q, hp=HP, step=1, seed=4)
    assert fg.sync_status() == 0
    assert torch.equal(loss.detach(), (losses * share).sum()) and torch.equal(x.grad.view(90, 128), dX)
    assert all(_same(a, b) for a, b in zip(head._layer("weight", 0)[:4], (W, m, v, q)))
    with torch.no_grad():
        t[:] = -100
        assert float(head(x, t)) == 0.0  # no token counts


def test_inputs_without_gradient_still_train():
    block, head = ForgeGatedMLP(64, 128, hp=HP), ForgeHeadLoss(64, 100, hp=HP, seed=3)
    old = [p.data.clone() for p in (block.gate, block.up, block.down, head.weight)]
    head(block(_x(40, 64)), torch.arange(40).cuda()).backward()
    assert fg.sync_status() == 0
    for p, o in zip((block.gate, block.up, block.down, head.weight), old):
        assert not torch.equal(p.data, o) and p.grad is None
    with pytest.raises(TypeError):
        block(_x(40, 64).float())
    with pytest.raises(TypeError):
        head(_x(40, 64).float(), torch.arange(40).cuda())
    with pytest.raises(ValueError):
        head(_x(40, 64), torch.arange(39).cuda())


@pytest.mark.parametrize("state", ["fp32", "bf16"])
def test_the_example_learns(state):
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_lm.py")
    spec = importlib.util.spec_from_file_location("gated_lm", path)
    gated_lm = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(gated_lm)
    losses = gated_lm.train(steps=60, state=state, show=None)
    # the uniform guess over 1003 tokens is 6.91; the permutation is learnt token by token
    assert 6.5 < losses[0] < 7.5 and losses[-1] < 2.0, losses
