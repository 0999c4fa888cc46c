"""The modules of blocks.py under another default type, and differentiated twice (needs a GB300)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
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
