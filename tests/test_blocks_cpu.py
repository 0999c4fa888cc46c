"""Construction of the modules of blocks.py (CPU only: no kernel is launched)."""
import pytest
import torch

from backward_optimizer_gb300.blocks import ForgeGatedMLP, ForgeHeadLoss, ForgeNorm


def test_parameters_and_states():
    n = ForgeNorm(8, device="cpu")
    assert n.weight.requires_grad and n.bias.requires_grad
    assert ForgeNorm(8, kind="rms", device="cpu").bias is None and ForgeNorm(8, bias=False, device="cpu").bias is None
    b = ForgeGatedMLP(64, 128, state="int8", device="cpu")
    assert b.gate.shape == (128, 64) and b.up.shape == (128, 64) and b.down.shape == (64, 128)
    assert not any(p.requires_grad for p in b.parameters())
    assert b.gate_m.dtype == torch.int8 and b.down_q.numel() == 2 * 64 * 128 // 64
    h = ForgeHeadLoss(64, 100, opt="lion", state="bf16", device="cpu")
    assert h.weight_m.dtype == torch.bfloat16 and h.weight_v is None and h.weight_q is None
    assert ForgeHeadLoss(64, 100, opt="sgd", device="cpu").weight_m is None
    # everything a checkpoint needs
    assert set(b.state_dict()) == {f"{w}{s}" for w in ("gate", "up", "down") for s in ("", "_m", "_v", "_q")}


@pytest.mark.parametrize("make", [lambda: ForgeNorm(8, kind="batch", device="cpu"),
                                  lambda: ForgeGatedMLP(64, 128, act="tanh", device="cpu"),
                                  lambda: ForgeGatedMLP(64, 128, opt="adam", device="cpu"),
                                  lambda: ForgeHeadLoss(64, 100, state="fp8", device="cpu")])
def test_refusals(make):
    with pytest.raises(ValueError):
        make()
