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
