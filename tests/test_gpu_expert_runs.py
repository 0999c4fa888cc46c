"""Products grouped by expert where a run itself is long (its own element numbers past 32 bits), where dX and the weights'
gradients share a launch, where units go in groups of four, and where tensors end with their memory; against the formulas in
binary64 (tolerances: operators_reference.py)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import test_gpu_gated as dense
from tests.operators_reference import F64, U8, acc, assert_close
from tests.test_gpu_experts import _backward, _full, _gated_inputs, _of, _offsets, _outside, _runs, _tensor
from tests.test_gpu_waits import _check as _check_waits
from tests.test_gpu_waits import _rand
from workloads import Hparams

pytestmark = pytest.mark.gpu

GRADIENT = dict(opt="sgd_momentum", hp=Hparams(lr=1.0, momentum=0.0, weight_decay=0.0), step=1)  # an FP32 m is the gradient


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


# The wide operand is zero but for rows at the run's start, around its bytes 2^31 and 2^32 and its element 2^32, and at its
# end; the other one is random everywhere, so that a row read at a wrong place shows.  Tiles of gradients on pairs (four
# experts) and on single CTAs (two); widths in blocks of 64 columns and not.
@pytest.mark.parametrize("wide, narrow, experts", [(8192, 64, 4), (8192, 256, 4), (8192, 64, 2), (8200, 72, 4)])
@pytest.mark.parametrize("wide_x", [True, False])
def test_a_run_past_32_bits(wide, narrow, experts, wide_x):
    sizes = [0, 530000, 3, 45] if experts == 4 else [530000, 45]
    R, E = sum(sizes), len(sizes)
    gen = torch.Generator("cuda").manual_seed(wide + narrow + experts)
    rows = torch.zeros(R, dtype=torch.bool, device="cuda")
    for at in (0, (1 << 30) // wide, (1 << 31) // wide, (1 << 32) // wide, 530000):
        rows[max(0, at - 12):at + 13] = True
    rows[530000:] = True
    big = torch.zeros(R, wide, dtype=torch.bfloat16, device="cuda")
    big[rows] = torch.randn(int(rows.sum()), wide, generator=gen, device="cuda").bfloat16()
    small = torch.randn(R, narrow, generator=gen, device="cuda").bfloat16()
    X, dY = (big, small) if wide_x else (small, big)
    (D, F), off = (X.shape[1], dY.shape[1]), _offsets(sizes)
    W = (torch.randn(E, F, D, generator=gen, device="cuda") * D ** -0.5).bfloat16()
    Y, dX, dW = _full(R, F), _full(R, D), _full(E, F, D)
    fg.expert_linear(X, W, off, Y)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    m = torch.full((E, F, D), 3.0, device="cuda")
    fg.expert_linear_backward_step(dY, X, W.clone(), off, None, m, None, None, **GRADIENT)
    assert fg.sync_status() == 0
    for e, r in _runs(sizes):
        if r.stop == r.start:
            assert not dW[e].any() and not m[e].any()
            continue
        at = torch.nonzero(rows[r])[:, 0] + r.start
        x, d, w = X[at].to(F64), dY[at].to(F64), W[e].to(F64)
        c = d.T @ x
        tol = acc(c, 16 * len(at))  # rows far apart: a step of the tensor core's sum for each
        assert_close(dW[e], c, U8 * c.abs() + (1 + U8) * tol, f"dW of expert {e}")
        assert_close(m[e], c, tol, f"m of expert {e}")
        for got, c, k, name in ((Y[at], x @ w.T, D, "Y"), (dX[at], d @ w, F, "dX")):
            assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), f"{name} of expert {e}")
    # rows whose wide operand is zero give zero
    assert not (Y if wide_x else dX)[~rows].any()


def _linear(sizes, lead, tail, D, F, seed):
    gen = torch.Generator().manual_seed(seed)
    R, E = lead + sum(sizes) + tail, len(sizes)
    X, dY, W = _tensor(gen, R, D), _tensor(gen, R, F), _tensor(gen, E, F, D, std=D ** -0.5)
    out = _outside(R, sizes, lead)
    X[out], dY[out] = float("nan"), float("inf")
    return X, dY, W, _offsets(sizes, lead), out


def _uneven(experts, mean, seed):
    """Lengths between 0 and twice the mean, some of them 0."""
    gen = torch.Generator().manual_seed(seed)
    n = [int(v) for v in torch.randint(0, 2 * mean + 1, (experts,), generator=gen)]
    for e in range(0, experts, 7):
        n[e] = 0
    return n


# dX and dW together.  On pairs: over 40 and under 256 rows an expert, and at least a tile of gradients for each of 76
# pairs (experts * tiles of 256 x 256); from 16 for each on, in groups of four.  On single CTAs: fewer tiles.
BOTH = [(_uneven(32, 70, 1), 2, 9, 520, 1032), (_uneven(40, 90, 2), 0, 0, 1024, 512), (_uneven(20, 200, 3), 1, 0, 264, 1288),
        (_uneven(96, 60, 4), 3, 40, 520, 1032), (_uneven(110, 48, 5), 0, 1, 1000, 776), (_uneven(90, 130, 6), 0, 0, 768, 1280),
        (_uneven(6, 90, 7), 1, 2, 136, 328), (_uneven(3, 130, 8), 0, 5, 512, 256)]


@pytest.mark.parametrize("case", range(len(BOTH)))
def test_gradients_in_one_launch(case):
    sizes, lead, tail, D, F = BOTH[case]
    X, dY, W, off, out = _linear(sizes, lead, tail, D, F, case)
    R, E = len(X), len(sizes)
    dX, dW, dX1, dW1 = _full(R, D), _full(E, F, D), _full(R, D), _full(E, F, D)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    fg.expert_linear_backward(dY, X, W, off, dX1, None)
    fg.expert_linear_backward(dY, X, W, off, None, dW1)
    assert fg.sync_status() == 0
    assert torch.equal(dW, dW1)
    for e, r in _runs(sizes, lead):
        if r.stop == r.start:
            assert not dW[e].any()
            continue
        x, d, w = X[r].to(F64), dY[r].to(F64), W[e].to(F64)
        for got, c, k, name in ((dX[r], d @ w, F, "dX"), (dX1[r], d @ w, F, "dX alone"), (dW[e], d.T @ x, r.stop - r.start, "dW")):
            assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), f"{name} of expert {e}")
    assert (dX[out] == 7.0).all() and (dX1[out] == 7.0).all()


@pytest.mark.parametrize("case", range(len(BOTH)))
def test_waits_of_one_launch(case):
    sizes, lead, tail, D, F = BOTH[case]
    X, dY, W, off, _ = _linear(sizes, lead, tail, D, F, case)
    dX, dW = torch.zeros_like(X), torch.zeros_like(W)
    fg.set_wait_limit_ns(20_000_000)
    try:
        _check_waits(lambda: fg.expert_linear_backward(dY, X, W, off, dX, dW), [dX, dW])
    finally:
        fg.set_wait_limit_ns(2_000_000_000)


# gradients of the gated block in groups of four: 16 tiles of 256 x 256 for each of 76 pairs, rows by expert under 256
@pytest.mark.parametrize("sizes, lead, tail, D, F", [(_uneven(32, 20, 11), 2, 3, 520, 1032), (_uneven(64, 100, 12), 0, 7, 512, 776),
                                                     (_uneven(200, 5, 13), 1, 0, 264, 520), ([0] * 31 + [300] + [0] * 38, 0, 0, 512, 768)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_gradients_in_groups(sizes, lead, tail, D, F, act):
    i = _gated_inputs(sizes, lead, tail, D, F, seed=14)
    dX, *dW = _backward(i, _offsets(sizes, lead), act)
    assert fg.sync_status() == 0
    for e, r in _runs(sizes, lead):
        if r.stop == r.start:
            assert not any(w[e].any() for w in dW)
            continue
        want, tol = dense._gradients(_of(i, e, r), act)
        for got, c, t, name in zip((dX[r], *(w[e] for w in dW)), want, tol, ("dX", "dWg", "dWu", "dWd")):
            assert_close(got, c, (1 + U8) * t + U8 * c.abs(), f"{name} of expert {e}")
    assert (dX[_outside(len(dX), sizes, lead)] == 7.0).all()


def _at_the_end(t):
    """t at the very end of an allocation of whole pages (44 MiB, a segment of its own)."""
    whole = torch.zeros(22 << 20, dtype=torch.bfloat16, device="cuda")
    v = whole[-t.numel():].view(t.shape)
    v.copy_(t)
    return v


# the linear layer's forward, backward (in one launch and in two) and step on tensors that end with their memory, runs
# shorter than a slice at the end: single CTAs, pairs, blocks of 64 columns and not (rows whose number leaves starts 32-byte aligned)
@pytest.mark.parametrize("sizes, D, F", [([82, 20, 0, 14], 520, 264), ([82, 20, 0, 13], 512, 256),
                                         (_uneven(32, 70, 1) + [13], 520, 1032), (_uneven(32, 70, 1) + [13], 512, 1024),
                                         ([300, 0, 400, 1], 512, 1024)])
def test_linear_on_tensors_that_end_with_their_memory(sizes, D, F):
    X, dY, W, off, _ = _linear(sizes, 0, 0, D, F, 9)
    X, dY, W = _at_the_end(X), _at_the_end(dY), _at_the_end(W)
    R, E = len(X), len(sizes)
    Y, dX, dX1 = (_at_the_end(_full(R, n)) for n in (F, D, D))
    dW, dW1 = _at_the_end(_full(E, F, D)), _at_the_end(_full(E, F, D))
    fg.expert_linear(X, W, off, Y)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    fg.expert_linear_backward(dY, X, W, off, dX1, None)
    fg.expert_linear_backward(dY, X, W, off, None, dW1)
    steps = []
    for state in (torch.float32, torch.bfloat16) + ((torch.int8,) if D % 64 == 0 else ()):
        m = torch.zeros(E, F, D, dtype=state, device="cuda")
        q = torch.zeros(2 * m.numel() // 64, device="cuda") if state is torch.int8 else None
        fg.expert_linear_backward_step(dY, X, W.clone(), off, None, m, None, q, **GRADIENT)
        steps.append(m)
    assert fg.sync_status() == 0
    assert torch.equal(dW, dW1)
    for e, r in _runs(sizes):
        if r.stop == r.start:
            assert not dW[e].any() and not any(m[e].any() for m in steps)
            continue
        x, d, w = X[r].to(F64), dY[r].to(F64), W[e].to(F64)
        for got, c, k, name in ((Y[r], x @ w.T, D, "Y"), (dX[r], d @ w, F, "dX"), (dX1[r], d @ w, F, "dX alone"),
                                (dW[e], d.T @ x, r.stop - r.start, "dW")):
            assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), f"{name} of expert {e}")
        c = d.T @ x
        assert_close(steps[0][e], c, acc(c, r.stop - r.start), f"m of expert {e}")
        # rounded stochastically: a whole step
        assert_close(steps[1][e], c, 2 * U8 * c.abs() + (1 + 2 * U8) * acc(c, r.stop - r.start), f"bf16 m of expert {e}")


def test_gated_step_on_tensors_that_end_with_their_memory():
    sizes, D, F = [82, 20, 57, 0, 10, 7, 0, 36, 110, 8, 237, 0, 2, 117, 237, 13], 520, 1032
    i = _gated_inputs(sizes, 0, 0, D, F, seed=15)
    i = {k: _at_the_end(v) for k, v in i.items()}
    E = len(sizes)
    m = [torch.zeros(E, *s, device="cuda") for s in ((F, D), (F, D), (D, F))]
    layers = [(i[n].clone(), s, None, None, k) for k, (n, s) in enumerate(zip(("Wg", "Wu", "Wd"), m))]
    dX = _at_the_end(_full(sum(sizes), D))
    fg.expert_gated_mlp_backward_step(i["dY"], i["X"], i["G"], i["U"], *layers, _offsets(sizes), dX, **GRADIENT)
    assert fg.sync_status() == 0
    for e, r in _runs(sizes):
        if r.stop == r.start:
            assert not any(s[e].any() for s in m)
            continue
        want, tol = dense._gradients(_of(i, e, r), "silu")
        assert_close(dX[r], want[0], (1 + U8) * tol[0] + U8 * want[0].abs(), f"dX of expert {e}")
        for s, c, t, name in zip(m, want[1:], tol[1:], ("dWg", "dWu", "dWd")):
            assert_close(s[e], c, t, f"{name} of expert {e}")
