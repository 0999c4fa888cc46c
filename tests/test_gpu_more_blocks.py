"""The modules of experts, dropout and preference loss: the same bits as the calls they are made of, their gradients, state
dicts, and a training step of all of them together; and the calls in graphs and on streams."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.blocks import (ForgeDropout, ForgeExpertMLP, ForgeHeadLoss, ForgeNorm, ForgePreferenceLoss)
from tests.operators_reference import F64, U8, act_both
from workloads import Hparams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


HP = Hparams(lr=1e-2)


def _rand(seed, *shape, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).bfloat16().cuda()


def _off(sizes, lead=0):
    return torch.tensor([lead] + sizes).cumsum(0).to(torch.int32).cuda()


def _twin(module, make):
    other = make()
    other.load_state_dict(module.state_dict())
    return other


@pytest.mark.parametrize("state", ["fp32", "bf16", "int8"])
def test_expert_module_is_its_calls(state):
    sizes, D, F = [20, 0, 33, 70], 128, 192
    off = _off(sizes, 2)
    make = lambda: ForgeExpertMLP(D, F, 4, act="gelu_tanh", hp=HP, state=state, seed=7)  # noqa: E731
    block = make()
    x = _rand(0, 130, D).requires_grad_()
    twin = _twin(block, make)
    with torch.no_grad():
        quiet = block(x, off)
    y = block(x, off)
    g = _rand(1, 130, D)
    y.backward(g)
    assert torch.equal(y, quiet) and not y[:2].any() and not y[125:].any()
    Y, G, U, dX = torch.zeros_like(y), *(torch.empty(130, F, dtype=y.dtype, device="cuda") for _ in range(2)), torch.zeros_like(y)
    fg.expert_gated_mlp(x.detach(), twin.gate.data, twin.up.data, twin.down.data, off, Y, G, U, act="gelu_tanh")
    fg.expert_gated_mlp_backward_step(g, x.detach(), G, U, twin._layer("gate", 7), twin._layer("up", 8), twin._layer("down", 9), off,
                                      dX, act="gelu_tanh", opt="adamw", hp=HP, step=1)
    assert torch.equal(y, Y) and torch.equal(x.grad, dX) and not dX[:2].any() and not dX[125:].any()
    for (k, a), b in zip(block.state_dict().items(), twin.state_dict().values()):
        if k != "step":
            assert torch.equal(a, b), k
    assert block.step == 2 and block.state_dict()["step"] == 2
    with pytest.raises(RuntimeError):  # one backward per forward
        y2 = block(x, off)
        y2.sum().backward(retain_graph=True)
        y2.sum().backward()
    # inputs that need no gradient: the weights are trained all the same
    before = block.gate.data.clone()
    block(x.detach(), off).backward(g)
    assert not torch.equal(before, block.gate.data)


def test_dropout_module():
    x, r = _rand(2, 40, 72).requires_grad_(), _rand(3, 40, 72).requires_grad_()
    drop = ForgeDropout(0.3, seed=11)
    y1, y2 = drop(x, residual=r), drop(x, residual=r)
    assert not torch.equal(y1, y2) and drop.step == 3
    want, dx = torch.empty_like(x), torch.empty_like(x)
    fg.dropout(x.detach(), want, 0.3, seed=11, step=2, residual=r.detach())
    g = _rand(4, 40, 72)
    y2.backward(g)
    fg.dropout_backward(g, dx, 0.3, seed=11, step=2)
    assert torch.equal(y2, want) and torch.equal(x.grad, dx) and torch.equal(r.grad, g)
    again = ForgeDropout(0.3, seed=11)
    again.load_state_dict(drop.state_dict())
    assert torch.equal(again(x), drop(x))
    drop.eval()
    assert torch.equal(drop(x), x) and torch.equal(drop(x, residual=r), x + r) and drop.step == 4
    # a view that is not contiguous
    t = x.detach().t()
    z = ForgeDropout(0.3, seed=11)(t)
    fg.dropout(t.contiguous(), dx.view(72, 40), 0.3, seed=11, step=1)
    assert torch.equal(z, dx.view(72, 40))


def test_head_without_reduction_and_preference_module():
    T, D, V = 90, 64, 300
    sizes = [20, 15, 30, 25]
    off = _off(sizes)
    make = lambda **kw: ForgeHeadLoss(D, V, hp=HP, seed=3, **kw)  # noqa: E731
    head = make(reduction="none")
    twin = _twin(head, make)
    x = _rand(5, T, D).requires_grad_()
    target = torch.randint(V, (T,), generator=torch.Generator().manual_seed(6)).cuda()
    target[::9] = -100
    mask = target != -100
    ref = torch.rand(T, generator=torch.Generator().manual_seed(7)).cuda() * 6
    nll = head(x, target)
    with torch.no_grad():
        assert torch.equal(head(x, target), nll)
        assert make(reduction="none")(x.view(9, 10, D), target.view(9, 10)).shape == (9, 10)
    pref = ForgePreferenceLoss(beta=0.2, smoothing=0.1, mean=True)
    loss, reward = pref(nll, ref, off, mask)
    assert not reward.requires_grad
    w = torch.tensor([0.3, 0.7], device="cuda")
    (loss * w).sum().backward()
    l2, r2, s2, dnll = torch.empty(2, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.empty(T, device="cuda")
    tl, lse, dX = torch.empty(T, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
    fg.linear_cross_entropy(x.detach(), twin.weight.data, target, tl, lse)
    fg.preference_loss(tl, ref, off, l2, r2, s2, mask=mask, beta=0.2, smoothing=0.1, mean=True)
    fg.preference_loss_backward(w, s2, off, dnll, mask=mask)
    W, m, v, q, seed = twin._layer("weight", 3)
    fg.linear_cross_entropy_step(x.detach(), W, target, lse, dnll, dX, m, v, q, opt="adamw", hp=HP, step=1, seed=3)
    assert torch.equal(nll, tl) and torch.equal(loss, l2) and torch.equal(reward, r2)
    assert torch.equal(x.grad, dX) and torch.equal(head.weight.data, W) and torch.equal(head.weight_m, m)


def test_gradients_cannot_be_differentiated():
    x, off = _rand(8, 12, 64).requires_grad_(), _off([5, 7])
    nll = torch.rand(12, device="cuda", requires_grad=True)
    for y in (ForgeExpertMLP(64, 64, 2, hp=HP)(x, off), ForgeDropout(0.5)(x), ):
        (g,) = torch.autograd.grad(y.float().sum(), x, create_graph=True)
        with pytest.raises(RuntimeError, match="cannot be differentiated"):
            g.float().sum().backward()
    (g,) = torch.autograd.grad(ForgePreferenceLoss()(nll, None, off)[0].sum(), nll, create_graph=True)
    with pytest.raises(RuntimeError, match="cannot be differentiated"):
        g.sum().backward()


def test_default_types_do_not_matter():
    x, off = _rand(9, 12, 64), _off([5, 7])
    try:
        torch.set_default_dtype(torch.float64)
        nll = torch.rand(12, dtype=torch.float32, device="cuda", requires_grad=True)
        loss, _ = ForgePreferenceLoss()(nll, None, off)
        loss.sum().backward()
        assert loss.dtype == torch.float32 and nll.grad.dtype == torch.float32
        ForgeExpertMLP(64, 64, 2, hp=HP)(x.requires_grad_(), off).sum().backward()
    finally:
        torch.set_default_dtype(torch.float32)


def test_refusals():
    with pytest.raises(ValueError):
        ForgeDropout(1.5)
    with pytest.raises(ValueError):
        ForgePreferenceLoss(kind="other")
    with pytest.raises(ValueError):
        ForgeExpertMLP(64, 64, 2, act="other")
    with pytest.raises(ValueError):
        ForgeHeadLoss(64, 64, reduction="sum")
    block, off = ForgeExpertMLP(64, 64, 2, hp=HP), _off([5, 7])
    x = _rand(10, 12, 64)
    for bad in (x.float(), x.view(1, 12, 64), x[:, :32]):
        with pytest.raises((TypeError, ValueError)):
            block(bad, off)
    for bad in (off.long(), off[:2], off.cpu()):
        with pytest.raises((TypeError, ValueError)):
            block(x, bad)
    with pytest.raises(ValueError):
        ForgePreferenceLoss()(torch.zeros(5, device="cuda"), None, torch.zeros(4, dtype=torch.int32, device="cuda"))


class _Model(torch.nn.Module):
    """embedding -> norm -> experts (two a token) -> dropout, residual -> norm -> head's token losses -> preference loss"""

    def __init__(self, vocab, D, F, E, seed):
        super().__init__()
        torch.manual_seed(seed)
        self.embed = torch.nn.Embedding(vocab, D, device="cuda", dtype=torch.bfloat16)
        self.norm1, self.norm2 = ForgeNorm(D, kind="rms"), ForgeNorm(D)
        self.experts = ForgeExpertMLP(D, F, E, hp=HP, seed=10)
        self.drop = ForgeDropout(0.1, seed=20)
        self.head = ForgeHeadLoss(D, vocab, hp=HP, seed=30, reduction="none")
        self.pref = ForgePreferenceLoss(beta=0.5, mean=True)

    def forward(self, tokens, target, route, ref, sequences, mask):
        x = self.embed(tokens)
        E = self.experts.gate.shape[0]
        order = torch.argsort(route.reshape(-1), stable=True)
        offsets = torch.searchsorted(route.reshape(-1)[order], torch.arange(E + 1, device="cuda")).to(torch.int32)
        rows = self.norm1(x)[order // 2]
        y = torch.zeros_like(x).index_add(0, order // 2, self.experts(rows, offsets) * 0.5)
        h = self.drop(y, residual=x)
        self.hidden = h
        return self.pref(self.head(self.norm2(h), target), ref, sequences, mask)


def test_a_training_step_of_all_of_them():
    """Forward against the formulas; backward: every gradient arrives, and the same step again gives the same bits."""
    V, D, F, E, T = 500, 128, 192, 6, 400
    gen = torch.Generator().manual_seed(0)
    tokens, target = torch.randint(V, (T,), generator=gen).cuda(), torch.randint(V, (T,), generator=gen).cuda()
    target[::11] = -100
    route = torch.stack([torch.randperm(E - 1, generator=gen)[:2] for _ in range(T)]).cuda()  # the last expert gets none
    ref = (torch.rand(T, generator=gen) * 8).cuda()
    seqs, mask = _off([120, 90, 100, 90]), target != -100
    results = []
    for _ in range(2):
        m = _Model(V, D, F, E, 1)
        w0 = {k: v.clone() for k, v in m.state_dict().items()}
        loss, reward = m(tokens, target, route, ref, seqs, mask)
        loss.mean().backward()
        assert fg.sync_status() == 0
        results.append([loss, reward, m.embed.weight.grad, m.norm1.weight.grad, m.norm2.weight.grad] + list(m.state_dict().values()))
        assert all(p.grad is not None and torch.isfinite(p.grad).all() and p.grad.any() for p in
                   (m.embed.weight, m.norm1.weight, m.norm2.weight, m.norm2.bias))
        assert not torch.equal(w0["experts.gate"][:5], m.experts.gate[:5]) and not torch.equal(w0["head.weight"], m.head.weight)
    # index_add in the sum of two experts' rows adds in any order: two terms, so its result does not depend on it
    assert all(torch.equal(a, b) for a, b in zip(*results) if torch.is_tensor(a))

    # the forward pass in binary64 from the block's own hidden rows (each stage against its input)
    with torch.no_grad():
        h = m.hidden.to(F64)
        mean = h.mean(1, keepdim=True)
        n2 = ((h - mean) / ((h - mean).square().mean(1, keepdim=True) + m.norm2.eps).sqrt()).bfloat16().to(F64)
        logits = n2 @ w0["head.weight"].to(F64).T
        nll = torch.logsumexp(logits, 1) - logits.gather(1, target.clamp_min(0)[:, None])[:, 0]
        d = torch.where(mask, ref.to(F64) - nll, 0.0)
        cuts = seqs.tolist()
        score = torch.stack([d[a:b].sum() / mask[a:b].sum() for a, b in zip(cuts, cuts[1:])])
        # hidden rows normed to bf16 carry half a step each; 0.5 (beta) times means of some 80 tokens' losses
        assert (reward.to(F64) - 0.5 * score).abs().max() < 0.5 * 2 * U8 * logits.abs().max()
        x = m.embed.weight[tokens].to(F64)
        xn = (x / (x.square().mean(1, keepdim=True) + m.norm1.eps).sqrt()).bfloat16().to(F64)
        y = torch.zeros_like(x)
        for t in range(0, T, 37):
            for e in route[t].tolist():
                g, u = w0["experts.gate"][e].to(F64) @ xn[t], w0["experts.up"][e].to(F64) @ xn[t]
                y[t] += 0.5 * (w0["experts.down"][e].to(F64) @ (act_both(g, "silu")[0] * u))
            kept = (m.hidden[t].to(F64) - x[t]).abs() > 0
            got = (m.hidden[t].to(F64) - x[t])[kept] * (65536 - 6554) / 65536
            # y's own roundings (H, each expert's row, their sum) and the sum with x, each half a step
            assert (got - y[t][kept]).abs().max() < 8 * U8 * (y[t].abs().max() + x[t].abs().max())


class _Calls:
    """Experts, dropout, preference loss, forward and backward, into buffers of their own."""

    def __init__(self, seed, sizes, D, F, P):
        R, E = sum(sizes), len(sizes)
        self.off, self.seqs = _off(sizes), _off([R // (2 * P)] * (2 * P))
        self.x, self.r = _rand(seed, R, D), _rand(seed + 1, R, D)
        self.Wg, self.Wu, self.Wd = _rand(seed + 2, E, F, D, std=0.05), _rand(seed + 3, E, F, D, std=0.05), _rand(seed + 4, E, D, F, std=0.05)
        self.nll, self.ref = _rand(seed + 5, R).float().abs(), _rand(seed + 6, R).float().abs()
        self.step = torch.tensor([5], device="cuda")
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        f = torch.float32
        self.out = {"Y": e(R, D), "G": e(R, F), "U": e(R, F), "z": e(R, D), "dz": e(R, D), "dx": e(R, D), "dWg": e(E, F, D),
                    "dWu": e(E, F, D), "dWd": e(E, D, F), "L": e(R, F), "loss": e(P, dt=f), "reward": e(2 * P, dt=f),
                    "slope": e(2 * P, dt=f), "dnll": e(R, dt=f)}

    def run(self, stream=None):
        o = self.out
        fg.expert_gated_mlp(self.x, self.Wg, self.Wu, self.Wd, self.off, o["Y"], o["G"], o["U"], stream=stream)
        fg.dropout(o["Y"], o["z"], 0.2, seed=3, step=self.step, residual=self.r, stream=stream)
        fg.preference_loss(self.nll, self.ref, self.seqs, o["loss"], o["reward"], o["slope"], stream=stream)
        fg.preference_loss_backward(o["loss"], o["slope"], self.seqs, o["dnll"], stream=stream)
        fg.dropout_backward(o["z"], o["dz"], 0.2, seed=3, step=self.step, stream=stream)
        fg.expert_gated_mlp_backward(o["dz"], self.x, o["G"], o["U"], self.Wg, self.Wu, self.Wd, self.off, o["dx"], o["dWg"], o["dWu"],
                                     o["dWd"], stream=stream)
        fg.expert_linear(self.x, self.Wg, self.off, o["L"], stream=stream)

    def copy(self):
        return {k: v.clone() for k, v in self.out.items()}

    def clear(self):
        for v in self.out.values():
            v.fill_(float("nan"))


def _all_equal(a, b):
    return all(torch.equal(a[k], b[k]) for k in a)


CALLS = [([3, 0, 40, 9], 128, 192, 2), ([300, 0, 500, 224], 512, 768, 8), ([1, 0, 1], 1024, 512, 1)]


def test_captured_and_replayed_with_other_sizes():
    """A captured pass reads offsets and step from the device at each replay."""
    for sizes, D, F, P in CALLS:
        c = _Calls(1, sizes, D, F, P)
        c.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        other = list(reversed(sizes))
        for s in (sizes, other, [sum(sizes)] + [0] * (len(sizes) - 1), sizes):
            c.off.copy_(_off(s))
            c.step += 1
            for k in ("Y", "G", "U"):
                c.out[k].zero_()
            c.run()
            want = c.copy()
            c.clear()
            g.replay()
            torch.cuda.synchronize()
            assert fg.sync_status() == 0
            assert _all_equal(c.copy(), want), s


def test_on_streams_at_once():
    """Two captured passes that replay at once, and eager calls on other streams, each with workspaces of its own."""
    calls = [_Calls(10 * i, *c) for i, c in enumerate(CALLS + CALLS[:1])]
    for c in calls:
        c.run()
    torch.cuda.synchronize()
    want = [c.copy() for c in calls]
    graphs = []
    for c in calls[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in calls]
    for c in calls:
        c.clear()
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        for c, s in zip(calls[2:], streams[2:]):
            c.run(stream=s)
    with torch.cuda.stream(streams[3]):
        calls[3].run()
    torch.cuda.synchronize()
    assert fg.sync_status() == 0
    assert all(_all_equal(c.copy(), w) for c, w in zip(calls, want))
