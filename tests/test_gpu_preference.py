"""The preference loss on the GPU against its formulas in binary64 (written out here) and against differences."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests.operators_reference import F64, assert_close

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _scores(nll, ref, sizes, lead, mask, mean):
    d = (0 if ref is None else ref.to(F64)) - nll.to(F64)
    out, per, at = [], [], lead
    for n in sizes:
        keep = torch.ones(n, dtype=torch.bool, device="cuda") if mask is None else mask[at:at + n]
        k = int(keep.sum())
        p = 1 / k if mean and k else 1.0
        out.append(d[at:at + n][keep].sum() * p)
        per.append(p)
        at += n
    return torch.stack(out), torch.tensor(per, dtype=F64, device="cuda")


def _loss(z, kind, beta, smoothing):
    ls = torch.nn.functional.logsigmoid
    if kind == "sigmoid":
        return -(1 - smoothing) * ls(z) - smoothing * ls(-z)
    return torch.relu(1 - z) if kind == "hinge" else ((z - 0.5) / beta) ** 2


def _inputs(sizes, lead, tail, seed, masked, spread=0.05):
    gen = torch.Generator().manual_seed(seed)
    T = lead + sum(sizes) + tail
    ref = torch.empty(T).exponential_(0.7, generator=gen)
    nll = ref + spread * torch.randn(T, generator=gen)
    mask = None
    if masked:
        mask = torch.rand(T, generator=gen) < 0.7
        bad = torch.tensor([float("nan"), float("inf"), float("-inf"), -3e38]).repeat(T)[:T]
        nll, ref = torch.where(mask, nll, bad), torch.where(mask, ref, bad.flip(0))
    out = torch.ones(T, dtype=torch.bool)
    out[lead:lead + sum(sizes)] = False
    nll[out] = float("nan")  # tokens of no sequence
    offsets = torch.tensor([lead] + sizes).cumsum(0).to(torch.int32)
    return [t if t is None else t.cuda() for t in (nll, ref, offsets, mask)]


def _ragged(pairs, most, seed):
    gen = torch.Generator().manual_seed(seed)
    return [int(n) for n in torch.randint(0, most + 1, (2 * pairs,), generator=gen)]


# sequences: single tokens, empty ones, around 32 tokens and chunks of 512, one that holds nearly all, many short, few
# long; one block's worth and many
CASES = [([1, 1], 0, 0), ([0, 5, 3, 0], 2, 3), ([31, 33, 32, 64], 0, 0), (_ragged(7, 700, 1), 5, 9), (_ragged(300, 4, 2), 0, 1),
         (_ragged(300, 0, 2), 0, 40), ([511, 513, 512, 1, 1024, 0], 0, 0), ([1, 20000, 3, 0, 2, 7], 11, 0),
         (_ragged(64, 60, 3), 0, 0), ([100003, 99999], 1, 2), (_ragged(40, 3000, 4), 0, 700), ([0, 0], 0, 0)]


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("kind, smoothing, margin", [("sigmoid", 0.0, 0.0), ("sigmoid", 0.1, 0.3), ("hinge", 0.0, -0.2),
                                                     ("ipo", 0.0, 0.0)])
@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("masked", [False, True])
def test_loss_and_gradient(case, kind, smoothing, margin, mean, masked):
    sizes, lead, tail = CASES[case]
    beta, P = 0.25, len(sizes) // 2
    nll, ref, offsets, mask = _inputs(sizes, lead, tail, case, masked)
    loss, reward, slope = (torch.full((n,), 9.0, device="cuda") for n in (P, 2 * P, 2 * P))
    fg.preference_loss(nll, ref, offsets, loss, reward, slope, mask=mask, beta=beta, kind=kind, smoothing=smoothing,
                       margin=margin, mean=mean)
    # the sums keep some 48 bits: their own rounding is far below that of binary32, into which the margin, z and each
    # result are rounded.  beta here is a power of two; the margin is taken as binary32 holds it
    score, per = _scores(nll, ref, sizes, lead, mask, mean)
    m = torch.tensor(margin, dtype=torch.float32).double().item()
    s = torch.tensor(smoothing, dtype=torch.float32).double().item()
    z = (beta * (score[:P] - score[P:]) - m).requires_grad_()
    want = _loss(z, kind, beta, s)
    g = torch.autograd.grad(want.sum(), z)[0]
    want = want.detach()
    # z is off by half a step and, through it, the loss by its slope; the steps after it (exponential, logarithm,
    # quotient: a few units in the last place of values up to 1 + |z|) by at most 16 EPS of them; ipo's slope
    # changes with z by 2 / beta^2
    zt = z.detach()
    step = EPS * zt.abs() + 4 * EPS
    if kind == "ipo":
        tol, gtol = step * g.abs() + 16 * EPS * want.abs() + step ** 2 / beta ** 2, step * 2 / beta ** 2 + 16 * EPS * g.abs()
    else:
        tol, gtol = step * g.abs() + 16 * EPS * want.abs() + 4 * EPS, step + 16 * EPS
    near = (zt - 1).abs() < step if kind == "hinge" else torch.zeros_like(zt, dtype=torch.bool)
    assert not near.any()
    assert_close(loss, want, tol, "loss")
    assert_close(reward, beta * score, 2 * EPS * (beta * score).abs() + 1e-12, "reward")
    ws = torch.cat([-g, g]) * beta * per
    assert_close(slope, ws, torch.cat([gtol, gtol]) * beta * per + 4 * EPS * ws.abs(), "slope")

    T = len(nll)
    dloss, dnll = torch.randn(P, generator=torch.Generator().manual_seed(1)).cuda(), torch.full((T,), 9.0, device="cuda")
    fg.preference_loss_backward(dloss, slope, offsets, dnll, mask=mask)
    want = torch.zeros(T, device="cuda")
    at = lead
    for i, n in enumerate(sizes):
        want[at:at + n] = slope[i] * dloss[i % P]
        at += n
    assert torch.equal(dnll, want if mask is None else torch.where(mask, want, 0.0))


def test_gradient_against_differences():
    sizes = [40, 7, 25, 60]
    nll, ref, offsets, mask = _inputs(sizes, 0, 0, 5, True)
    dloss = torch.tensor([0.3, -1.2], device="cuda")
    for kind in ("sigmoid", "ipo"):
        def total(x):
            score, _ = _scores(x, ref, sizes, 0, mask, True)
            z = 0.5 * (score[:2] - score[2:])
            return (_loss(z, kind, 0.5, 0.0) * dloss.double()).sum()
        loss, slope, dnll = torch.empty(2, device="cuda"), torch.empty(4, device="cuda"), torch.empty(len(nll), device="cuda")
        fg.preference_loss(nll, ref, offsets, loss, None, slope, mask=mask, beta=0.5, kind=kind, mean=True)
        fg.preference_loss_backward(dloss, slope, offsets, dnll, mask=mask)
        for t in torch.arange(0, len(nll), 9).tolist():
            if not mask[t]:
                assert dnll[t] == 0
                continue
            h = 1e-3
            up, down = nll.double().clone(), nll.double().clone()
            up[t] += h
            down[t] -= h
            d = ((total(up) - total(down)) / (2 * h)).item()
            assert abs(dnll[t].item() - d) < 1e-5 * max(1.0, abs(d))


def test_large_scores_keep_their_digits():
    """Sums of 10^5 tokens that nearly cancel between model and reference, and pairs far from the border."""
    n = 100000
    ref = torch.empty(2 * n).exponential_(0.2, generator=torch.Generator().manual_seed(6)).cuda()
    nll = ref.clone()
    nll[:n] += 2.0 ** -20
    offsets = torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    loss, reward = torch.empty(1, device="cuda"), torch.empty(2, device="cuda")
    fg.preference_loss(nll, ref, offsets, loss, reward, None, beta=1.0)
    want = -(nll.double() - ref.double())[:n].sum()
    assert abs(reward[0].item() - want.item()) <= 2 * EPS * abs(want.item()) and reward[1].item() == 0
    for shift, far in ((1.0, 0.0), (-1.0, 1e5)):
        nll = ref.double()
        nll[:n] -= shift
        nll = nll.float()
        fg.preference_loss(nll, ref, offsets, loss, reward, None, beta=1.0)
        d = (ref.double() - nll.double())[:n].sum().item()
        assert abs(loss.item() - (0.0 if shift > 0 else -d)) <= 4 * EPS * abs(d)


def test_a_pair_that_is_not_finite_stays_by_itself():
    sizes = [50, 60, 70, 40, 30, 20]
    nll, ref, offsets, _ = _inputs(sizes, 0, 0, 7, False)
    clean, slope = torch.empty(3, device="cuda"), torch.empty(6, device="cuda")
    fg.preference_loss(nll, ref, offsets, clean, None, slope)
    nll[55] = float("nan")  # chosen sequence 1
    loss, slope2 = torch.empty(3, device="cuda"), torch.empty(6, device="cuda")
    for kind in ("sigmoid", "hinge", "ipo"):
        fg.preference_loss(nll, ref, offsets, loss, None, slope2, kind=kind)
        assert loss.isnan().tolist() == [False, True, False]
        assert slope2.isnan().tolist() == [False, True, False, False, True, False]
    fg.preference_loss(nll, ref, offsets, loss, None, slope2)
    assert torch.equal(loss[[0, 2]], clean[[0, 2]]) and torch.equal(slope2[[0, 2, 3, 5]], slope[[0, 2, 3, 5]])


def test_offsets_out_of_range_stay_inside():
    """Unspecified results, but nothing outside the tensors is touched and the call ends."""
    T, P = 3000, 3
    for given in ([-7, 50, 20, 10**9, 5, 2**31 - 1, -1], [5, 4, 3, 2, 1, 0, -1], [9000] * 7):
        nll = torch.zeros(T + 64, device="cuda")
        offsets = torch.tensor(given, dtype=torch.int32, device="cuda")
        loss, slope, dnll = torch.empty(P, device="cuda"), torch.zeros(2 * P, device="cuda"), torch.full((T + 64,), 4.0, device="cuda")
        fg.preference_loss(nll[:T], None, offsets, loss, None, slope)
        fg.preference_loss_backward(loss, slope, offsets, dnll[:T])
        assert fg.sync_status() == 0
        assert (dnll[T:] == 4).all()


def test_no_pairs_and_no_tokens():
    e, off = torch.empty(0, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dnll = torch.full((40,), 2.0, device="cuda")
    fg.preference_loss(dnll, None, off, e)
    fg.preference_loss_backward(e, e, off, dnll)
    assert not dnll.any()
    loss = torch.empty(2, device="cuda")
    fg.preference_loss(e, None, torch.zeros(5, dtype=torch.int32, device="cuda"), loss, kind="hinge")
    assert torch.equal(loss, torch.ones(2, device="cuda"))
