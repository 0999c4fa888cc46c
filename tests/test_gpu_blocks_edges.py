"""The modules of blocks.py under another default type, and going on from a saved state (needs a GB300)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.autograd import ForgeLinear
from backward_optimizer_gb300.blocks import ForgeGatedMLP, ForgeHeadLoss, ForgeNorm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


@pytest.mark.parametrize("default", [torch.bfloat16, torch.float64])
@pytest.mark.parametrize("state", ["fp32", "int8"])
def test_any_default_type(default, state):
    x = torch.randn(40, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    t = torch.arange(40, device="cuda")
    w = [torch.randn(s, generator=torch.Generator().manual_seed(2)).bfloat16() * 0.02 for s in ((128, 64), (128, 64), (64, 128), (100, 64))]

    def step():
        n, block, head = ForgeNorm(64), ForgeGatedMLP(64, 128, state=state), ForgeHeadLoss(64, 100, state=state, seed=3)
        for p, value in zip((block.gate, block.up, block.down, head.weight), w):
            p.data.copy_(value)
        loss = head(block(n(x), residual=x), t)
        loss.backward()
        assert fg.sync_status() == 0
        return [loss.detach(), n.weight.grad, n.bias.grad, *block.state_dict().values(), *head.state_dict().values()]

    want = step()
    torch.set_default_dtype(default)
    try:
        got = step()
    finally:
        torch.set_default_dtype(torch.float32)
    assert [a.dtype for a in got] == [b.dtype for b in want]
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("state", ["fp32", "bf16", "int8"])
def test_training_goes_on_from_a_saved_state(state, tmp_path):
    """Two steps, a save, a load into new modules and one step: the bits of three steps."""
    hp = dict(lr=1e-2, weight_decay=0.01)

    def make():
        return torch.nn.ModuleDict({"block": ForgeGatedMLP(64, 128, state=state, hp=hp), "norm": ForgeNorm(64),
                                    "linear": ForgeLinear(64, 64, state=state, hp=hp, seed=7),
                                    "head": ForgeHeadLoss(64, 100, state=state, hp=hp, seed=3)})

    def step(m, i):
        x = torch.randn(40, 64, generator=torch.Generator().manual_seed(i)).bfloat16().cuda()
        m["head"](m["linear"](m["block"](m["norm"](x), residual=x)), torch.arange(40, device="cuda")).backward()

    a = make()
    for i in range(2):
        step(a, i)
    torch.save(a.state_dict(), tmp_path / "state")
    b = make()
    b.load_state_dict(torch.load(tmp_path / "state"))
    step(a, 2)
    step(b, 2)
    assert fg.sync_status() == 0
    want, got = a.state_dict(), b.state_dict()
    assert want.keys() == got.keys() and int(got["block.step"]) == 4
    assert all(torch.equal(want[k], got[k]) for k in want)
