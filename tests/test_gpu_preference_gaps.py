"""The preference loss over sequences with many empty ones between them, and over more tokens than chunks of the usual size
take: losses that are multiples of 2^-10, whose sums are exact in the kernel's pairs of binary32, so that the rewards are
those sums rounded once."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests.operators_reference import F64, assert_close

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24
BETA = 0.25  # a power of two: products by it are exact


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _check(sizes, lead, tail, masked, mean, seed):
    """sizes: a tensor of 2 P lengths, on the device.  Returns the milliseconds of forward and backward."""
    gen = torch.Generator("cuda").manual_seed(seed)
    P, T = len(sizes) // 2, lead + int(sizes.sum()) + tail
    offsets = torch.cat([sizes.new_zeros(1), sizes.cumsum(0)]).add(lead).to(torch.int32)
    nll, ref = (torch.randint(1024, (T,), generator=gen, device="cuda").float() / 1024 for _ in range(2))
    mask = torch.rand(T, generator=gen, device="cuda") < 0.7 if masked else None
    counts = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask
    seq = torch.repeat_interleave(torch.arange(2 * P, device="cuda"), sizes)
    inside = slice(lead, T - tail)
    # whole numbers: their sums in binary64 are exact in any order
    d = torch.where(counts, (ref.to(F64) - nll.to(F64)) * 1024, 0.0)[inside]
    total = torch.zeros(2 * P, dtype=F64, device="cuda").index_add_(0, seq, d) / 1024
    n = torch.zeros(2 * P, dtype=F64, device="cuda").index_add_(0, seq, counts[inside].to(F64))
    nll[:lead], nll[T - tail:] = float("nan"), float("nan")

    loss, reward, slope = (torch.full((k,), 9.0, device="cuda") for k in (P, 2 * P, 2 * P))
    dloss, dnll = torch.randn(P, generator=gen, device="cuda"), torch.full((T,), 9.0, device="cuda")
    at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    at[0].record()
    fg.preference_loss(nll, ref, offsets, loss, reward, slope, mask=mask, beta=BETA, kind="hinge", mean=mean)
    fg.preference_loss_backward(dloss, slope, offsets, dnll, mask=mask)
    at[1].record()
    assert fg.sync_status() == 0

    score = total / n.clamp_min(1) if mean else total
    if mean:  # a quotient of exact numbers: some 2^-46 before it is rounded
        assert_close(reward, BETA * score, 1.001 * EPS * (BETA * score).abs(), "reward")
    else:
        assert torch.equal(reward, (BETA * score).float())
    z = BETA * (score[:P] - score[P:])
    # z is off by half a step (mean: of each score's quotient too, some 2^-46); 1 - z once more
    tol = 1.001 * EPS * z.abs() + EPS * (1 - z).abs()
    assert_close(loss, (1 - z).clamp_min(0), tol, "loss")
    g = torch.where(z < 1, -1.0, 0.0)
    sure = ((z - 1).abs() > 2 * EPS).repeat(2)
    per = (1 / n.float().clamp_min(1)) if mean else torch.ones(2 * P, device="cuda")
    want = torch.cat([-g, g]).float() * BETA * per
    assert sure.double().mean() > 0.99 and torch.equal(slope[sure], want[sure])
    out = torch.zeros(T, device="cuda")
    out[inside] = (slope * dloss.repeat(2))[seq]
    assert torch.equal(dnll, torch.where(counts, out, 0.0))
    return at[0].elapsed_time(at[1])


def _lengths(n, full):
    """n sequences, all empty but those that `full` gives by their place."""
    sizes = torch.zeros(n, dtype=torch.int64, device="cuda")
    sizes[torch.tensor(list(full), device="cuda")] = torch.tensor(list(full.values()), device="cuda")
    return sizes


@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("pairs", [40, 70, 5000, 1 << 20, 1 << 24])
def test_empty_sequences_in_between(pairs, masked):
    """Neighbouring tokens that belong to sequences any number apart; empty ones at both ends."""
    n = 2 * pairs
    full = {3: 1, 5: 1, 6: 70, n // 3: 1, n // 3 + 1: 2, n // 2: 300, n - 9: 33, n - 7: 1}
    _check(_lengths(n, full), 2, 3, masked, False, pairs)
    elapsed = min(_check(_lengths(n, full), 0, 0, masked, False, pairs) for _ in range(2))
    # one by one, 2^25 of them would take seconds
    assert elapsed < 250
    _check(_lengths(n, {0: 20, n - 1: 20}), 0, 0, masked, False, pairs)
    _check(_lengths(n, {n // 2: 1}), 40, 40, masked, False, pairs)


@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("sizes", [
    [127, 128, 129, 130, 255, 256, 257, 1], [128] * 6, [384, 1, 127, 640], [1000, 1000, 1048, 1048],  # one block, chunks of 128
    [255, 256, 257, 511, 512, 513, 1, 9000], [256] * 40, [4097, 0, 1, 2],                             # many, chunks of 256
    [31, 32, 33, 63, 64, 65, 0, 1] * 40, [32] * 400,                                                  # chunks of 32 and 64
    [(1 << 21) + 5, (1 << 20) - 3, 0, 77], [(1 << 22) + 11, 1], [1 << 20] * 4,                        # chunks of 512
    [(1 << 24) + 3, 12345, 1 << 23, 513],                                                             # and of 4096
])
def test_around_chunks(sizes, masked, mean):
    _check(torch.tensor(sizes, device="cuda"), 1, 2, masked, mean, len(sizes))


def test_offsets_out_of_order_end_soon():
    """Unspecified results, but in bounded time and inside the tensors, also where millions of them go up and down."""
    P, T = 1 << 22, 4000
    for pattern in ([5, 4], [0, T], [T, 0], [T // 2, T // 2, 3]):
        offsets = torch.tensor(pattern, dtype=torch.int32, device="cuda").repeat(2 * P // len(pattern) + 1)[:2 * P + 1].contiguous()
        if len(offsets) < 2 * P + 1:
            offsets = torch.cat([offsets, offsets[:2 * P + 1 - len(offsets)]])
        nll, loss, slope = torch.zeros(T, device="cuda"), torch.empty(P, device="cuda"), torch.zeros(2 * P, device="cuda")
        dnll = torch.full((T + 64,), 4.0, device="cuda")
        at = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
        at[0].record()
        fg.preference_loss(nll, None, offsets, loss, None, slope)
        fg.preference_loss_backward(loss, slope, offsets, dnll[:T])
        at[1].record()
        assert fg.sync_status() == 0
        assert (dnll[T:] == 4).all() and at[0].elapsed_time(at[1]) < 250
