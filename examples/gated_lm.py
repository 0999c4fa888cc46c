"""Trains a small attention-free language model whose matrices are updated inside the backward pass.

    embedding -> [x + gated block(norm(x))] x layers -> norm -> head and loss

The gated blocks and the head (backward_optimizer_gb300.blocks) update their matrices and optimizer
states while the gradients pass through them; the norms' vectors and the embedding have ordinary
gradients and an ordinary optimizer.  Data: sequences in which the next token follows from the
present one by a fixed random permutation, with a tenth of the positions not counted in the loss.

The moments are binary32 or bfloat16.  INT8 second moments do not suit AdamW at this learning rate: an
element whose squared gradient is below 1/254 of its block's largest decodes to zero, and its step, divided
by the root of one step's share alone, grows up to thirtyfold.

    python examples/gated_lm.py [--steps 60] [--width 512] [--d-ff 1408] [--layers 2] [--vocab 1003]
"""
import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import backward_optimizer_gb300 as fg  # noqa: E402
from backward_optimizer_gb300.blocks import ForgeGatedMLP, ForgeHeadLoss, ForgeNorm  # noqa: E402


class Model(torch.nn.Module):
    def __init__(self, vocab, width, d_ff, layers, hp, state="fp32"):
        super().__init__()
        self.embedding = torch.nn.Embedding(vocab, width, device="cuda")
        # each block's three matrices take three consecutive rounding seeds, the head the next one
        self.norms = torch.nn.ModuleList(ForgeNorm(width, kind="rms") for _ in range(layers))
        self.blocks = torch.nn.ModuleList(ForgeGatedMLP(width, d_ff, hp=hp, state=state, seed=3 * i) for i in range(layers))
        self.final = ForgeNorm(width)
        self.head = ForgeHeadLoss(width, vocab, hp=hp, state=state, seed=3 * layers)

    def forward(self, tokens, target):
        x = self.embedding(tokens).to(torch.bfloat16)
        for norm, block in zip(self.norms, self.blocks):
            x = block(norm(x), residual=x)
        return self.head(self.final(x), target)


def train(steps=60, vocab=1003, width=512, d_ff=1408, layers=2, batch=(8, 256), state="fp32", seed=0, show=print):
    """The loss before each step, and the loss of the trained model without gradients at the end."""
    torch.manual_seed(seed)
    model = Model(vocab, width, d_ff, layers, hp=dict(lr=3e-3, weight_decay=0.0), state=state)
    other = torch.optim.AdamW([p for p in model.parameters() if p.requires_grad], lr=3e-3, weight_decay=0.0)
    follows = torch.randperm(vocab, device="cuda")
    losses, began = [], time.perf_counter()
    for step in range(steps + 1):
        tokens = torch.randint(vocab, batch, device="cuda")
        target = follows[tokens]
        target[torch.rand(batch, device="cuda") < 0.1] = model.head.ignore_index
        if step == steps:
            with torch.no_grad():
                losses.append(float(model(tokens, target)))
            break
        loss = model(tokens, target)
        other.zero_grad(set_to_none=True)
        loss.backward()
        other.step()
        losses.append(float(loss.detach()))
        if show and step % 10 == 0:
            show(f"step {step:4d}  loss {losses[-1]:.4f}")
    if fg.sync_status() != 0:
        raise RuntimeError("a bounded wait ran out on the device")
    if show:
        show(f"after {steps} steps  loss {losses[-1]:.4f}  ({(time.perf_counter() - began) / max(steps, 1) * 1e3:.2f} ms a step)")
    return losses


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("steps", 60), ("vocab", 1003), ("width", 512), ("d-ff", 1408), ("layers", 2)):
        ap.add_argument(f"--{name}", type=int, default=value)
    ap.add_argument("--state", choices=("fp32", "bf16"), default="fp32")
    a = ap.parse_args()
    fg.build()
    train(a.steps, a.vocab, a.width, a.d_ff, a.layers, state=a.state)
