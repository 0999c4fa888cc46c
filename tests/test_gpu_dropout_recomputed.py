"""ForgeDropout in regions whose forward the backward pass computes again: the same bits as without."""
import pytest
import torch
from torch.utils.checkpoint import checkpoint

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.blocks import ForgeDropout, ForgeGatedMLP, ForgeNorm
from workloads import Hparams

pytestmark = pytest.mark.gpu

HP = Hparams(lr=1e-2)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _rand(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


@pytest.mark.parametrize("reentrant", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_mask_of_the_gradient_is_the_mask_of_the_output(reentrant, dtype):
    drop = ForgeDropout(0.5, seed=1)
    x = _rand(0, 64, 257, dtype=dtype).abs().add(0.5).requires_grad_()
    y = checkpoint(lambda t: drop(t).square(), x, use_reentrant=reentrant)
    other = checkpoint(lambda t: drop(t).square(), x, use_reentrant=reentrant)
    assert not torch.equal(y == 0, other == 0)
    y.sum().backward()
    assert torch.equal(x.grad == 0, y == 0)
    assert drop.step == 3


@pytest.mark.parametrize("reentrant", [True, False])
def test_a_block_in_a_region(reentrant):
    """norm -> gated block -> dropout with its residual -> norm, twice, two steps: plain and recomputed."""
    def made():
        torch.manual_seed(3)
        return [ForgeNorm(128), ForgeGatedMLP(128, 192, hp=HP, seed=10), ForgeDropout(0.3, seed=20), ForgeNorm(128, kind="rms")]

    def region(m):
        return lambda x: m[3](m[2](m[1](m[0](x)), residual=x))

    results = []
    for recomputed in (False, True):
        layers = [made(), made()]
        got = []
        for step in range(2):
            x = _rand(step, 100, 128).requires_grad_()
            h = x
            for m in layers:
                h = checkpoint(region(m), h, use_reentrant=reentrant) if recomputed else region(m)(h)
            h.backward(_rand(7 + step, 100, 128))
            assert fg.sync_status() == 0
            got += [h.detach(), x.grad]
        for m in layers:
            for module in m:
                got += [p.grad for p in module.parameters() if p.grad is not None]
                got += [t for t in module.state_dict().values()]
        results.append(got)
    assert len(results[0]) == len(results[1])
    assert all(torch.equal(a, b) for a, b in zip(*results))


def test_a_captured_training_step_takes_a_mask_at_each_replay():
    """Forward and backward through the module in one graph, with the step on the device moved at its end."""
    drop, step = ForgeDropout(0.5, seed=4), torch.tensor([1], device="cuda")
    values, r = _rand(1, 40, 129).abs() + 0.5, _rand(2, 40, 129)

    def once(x, at):
        y = drop(x, residual=r, step=at)
        z = (y - r).square()
        return y.detach(), torch.autograd.grad(z.sum(), x)[0]

    once(values.clone().requires_grad_(), step)
    torch.cuda.synchronize()
    x = values.clone().requires_grad_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, dx = once(x, step)
        step += 1
    masks = []
    for k in (1, 2, 3):
        g.replay()
        torch.cuda.synchronize()
        assert fg.sync_status() == 0 and step.item() == k + 1
        want_y, want_dx = once(values.clone().requires_grad_(), k)
        assert torch.equal(y, want_y) and torch.equal(dx, want_dx)
        masks.append(dx != 0)
    assert not torch.equal(masks[0], masks[1]) and not torch.equal(masks[1], masks[2])
    assert drop.step == 1
