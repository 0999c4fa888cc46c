"""The modules' tensors and autograd on the CPU, with torch code in place of the library's calls (no kernel
runs here)."""
import pytest
import torch

from backward_optimizer_gb300 import blocks
from backward_optimizer_gb300.autograd import ForgeLinear
from backward_optimizer_gb300.blocks import ForgeGatedMLP, ForgeHeadLoss, ForgeNorm


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64])
def test_types_do_not_follow_the_default_type(default):
    torch.set_default_dtype(default)
    try:
        made = [ForgeNorm(8, device="cpu"), ForgeGatedMLP(64, 128, state="int8", device="cpu"),
                ForgeHeadLoss(64, 100, state="fp32", device="cpu"), ForgeLinear(64, 128, state="int8", device="cpu")]
    finally:
        torch.set_default_dtype(torch.float32)
    want = [ForgeNorm(8, device="cpu"), ForgeGatedMLP(64, 128, state="int8", device="cpu"),
            ForgeHeadLoss(64, 100, state="fp32", device="cpu"), ForgeLinear(64, 128, state="int8", device="cpu")]
    for a, b in zip(made, want):
        assert {k: v.dtype for k, v in a.state_dict().items()} == {k: v.dtype for k, v in b.state_dict().items()}


@pytest.fixture
def on_cpu(monkeypatch):
    """Formulas in place of the library's calls."""
    def layer_norm(x, w, b, y, mean=None, rstd=None, eps=1e-5, kind="layer", stream=None):
        m = x.mean(1)
        r = 1 / ((x - m[:, None]).square().mean(1) + eps).sqrt()
        mean.copy_(m)
        rstd.copy_(r)
        y.copy_((x - m[:, None]) * r[:, None] * w + b)

    def layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db=None, add=None, kind="layer", stream=None):
        xh = (x - mean[:, None]) * rstd[:, None]
        g = dy * w
        dx.copy_((g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * rstd[:, None])
        dw.copy_((dy * xh).sum(0))
        db.copy_(dy.sum(0))

    def gated_mlp(X, Wg, Wu, Wd, Y, G=None, U=None, residual=None, act="silu", stream=None):
        Y.copy_(X if residual is None else X + residual)

    def gated_step(dY, X, G, U, gate, up, down, dX=None, **kw):
        if dX is not None:
            dX.copy_(dY)

    def loss(X, W, target, out, lse, ignore_index=-100, stream=None):
        out.copy_(X.float().sum(1))
        lse.zero_()

    def loss_step(X, W, target, lse, dloss, dX=None, m=None, v=None, q=None, **kw):
        dX.copy_(dloss[:, None].expand_as(dX))

    for name, f in (("layer_norm", layer_norm), ("layer_norm_backward", layer_norm_backward), ("gated_mlp", gated_mlp),
                    ("gated_mlp_backward_step", gated_step), ("linear_cross_entropy", loss),
                    ("linear_cross_entropy_step", loss_step)):
        monkeypatch.setattr(blocks.ops, name, f)


# the norm's output used as it is (the incoming gradient needs no gradient), and through a function of its own
@pytest.mark.parametrize("use", [lambda y: y.sum(), lambda y: (y ** 3).sum()])
def test_a_second_derivative_raises(on_cpu, use):
    x = torch.randn(4, 8, generator=torch.Generator().manual_seed(0)).requires_grad_(True)
    n = ForgeNorm(8, device="cpu")
    (g,) = torch.autograd.grad(use(n(x)) + (x ** 4).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="ForgeNorm: the gradient cannot be differentiated"):
        g.square().sum().backward()
    # a first derivative, with and without create_graph, is the formula's
    y = torch.nn.functional.layer_norm(x, (8,), n.weight, n.bias)
    (want,) = torch.autograd.grad(use(y) + (x ** 4).sum(), x)
    (again,) = torch.autograd.grad(use(n(x)) + (x ** 4).sum(), x)
    assert torch.allclose(g, want, atol=1e-5) and torch.equal(g.detach(), again) and not again.requires_grad


def test_a_second_derivative_through_trained_modules_raises(on_cpu):
    x = torch.randn(4, 64, generator=torch.Generator().manual_seed(0)).bfloat16()
    for make, what in ((lambda: (lambda m, a: m(a).float().sum(), ForgeGatedMLP(64, 64, device="cpu")), "ForgeGatedMLP"),
                       (lambda: (lambda m, a: m(a, torch.zeros(4, dtype=torch.int64)), ForgeHeadLoss(64, 9, device="cpu")),
                        "ForgeHeadLoss")):
        call, m = make()
        a = x.clone().requires_grad_(True)
        (g,) = torch.autograd.grad(call(m, a) + (a.float() ** 2).sum(), a, create_graph=True)
        with pytest.raises(RuntimeError, match=f"{what}: the gradient cannot be differentiated"):
            g.float().square().sum().backward()


@pytest.mark.filterwarnings("ignore:Using backward")
def test_a_residual_keeps_its_graph(on_cpu):
    block = ForgeGatedMLP(64, 64, device="cpu")
    x, r = torch.zeros(4, 64).bfloat16(), torch.ones(4, 64).bfloat16().requires_grad_(True)
    (g,) = torch.autograd.grad((block(x, residual=r).float() ** 2).sum(), r, create_graph=True)
    assert torch.equal(g, 2 * torch.ones_like(g))
    block(x).float().sum().backward(create_graph=True)  # no gradient at all


def test_a_second_derivative_through_forge_linear_raises(monkeypatch):
    from backward_optimizer_gb300 import autograd
    monkeypatch.setattr(autograd, "linear_backward", lambda dY, X, W, m, v, q, dX, *a: dX.copy_(dY @ W))
    layer = ForgeLinear(64, 32, device="cpu")
    x = torch.randn(4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().requires_grad_(True)
    (g,) = torch.autograd.grad(layer(x).float().sum() + (x.float() ** 2).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="ForgeLinear: the gradient cannot be differentiated"):
        g.float().square().sum().backward()


@pytest.mark.parametrize("make", [lambda: ForgeLinear(64, 32, device="cpu"), lambda: ForgeGatedMLP(64, 128, device="cpu"),
                                  lambda: ForgeHeadLoss(64, 100, state="int8", device="cpu")])
def test_the_step_is_part_of_the_state(make, tmp_path):
    def model():
        return torch.nn.ModuleDict({"a": make(), "b": make()})
    m = model()
    assert not any(k.endswith("step") for k in m.state_dict())
    m["a"].step = 7
    m["a"]._pending = 7
    with torch.device("meta"):  # whatever the default device is, the step is a number on the host
        assert int(m.state_dict()["a.step"]) == 7
    torch.save(m.state_dict(), tmp_path / "s")
    for state in (torch.load(tmp_path / "s"), {k: v.clone() for k, v in m.state_dict().items()}):
        n = model()
        n["b"].step = 3
        n["a"]._pending = 1
        n.load_state_dict(state)  # strict
        assert n["a"].step == 7 and n["b"].step == 1 and type(n["a"].step) is int
        assert n["a"]._pending is None
    # a fresh state resets, and one saved before the step was part of it leaves the step to the caller
    m.load_state_dict(model().state_dict())
    assert m["a"].step == 1
    old = model().state_dict()
    for k in old._metadata:
        old._metadata[k] = {"version": 1}
    m["a"].step = 9
    m.load_state_dict(old)
    assert m["a"].step == 9
    with pytest.raises(RuntimeError, match="nexpected key"):
        m.load_state_dict({**old, "a.other": torch.zeros(1)})
