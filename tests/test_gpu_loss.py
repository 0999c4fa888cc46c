"""The cross entropy of a linear head on the GPU against its formulas in binary64 (operators_reference.py)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import operators_reference as ref
from tests.operators_reference import F64, U8, acc, assert_close, rounded
from workloads import Hparams

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _inputs(T, V, D, seed=0, spread=1.0, ignored=0.1):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=gen, device="cuda") * spread / D ** 0.5).bfloat16()
    t = torch.randint(V, (T,), generator=gen, device="cuda")
    t[torch.rand(T, generator=gen, device="cuda") < ignored] = IGNORE
    dloss = torch.rand(T, generator=gen, device="cuda") / max(T, 1)
    return x, w, t, dloss


def _forward(x, w, t, ignore=IGNORE, stream=None):
    loss, lse = (torch.full((x.shape[0],), 9.0, device="cuda") for _ in range(2))
    fg.linear_cross_entropy(x, w, t, loss, lse, ignore_index=ignore, stream=stream)
    return loss, lse


def _backward(x, w, t, lse, dloss, dx=True, dw=True, ignore=IGNORE):
    dX, dW = (torch.full_like(v, float("nan")) if on else None for v, on in ((x, dx), (w, dw)))
    fg.linear_cross_entropy_backward(x, w, t, lse, dloss, dX, dW, ignore_index=ignore)
    return dX, dW


def _check(x, w, t, dloss, loss, lse, dX, dW, ignore=IGNORE, scaled=True):
    X, W, DL = x.to(F64), w.to(F64), dloss.to(F64)
    T, D = X.shape
    V = W.shape[0]
    want, wlse, g, logits = ref.loss_and_gradient(X, W, t, DL, ignore)
    el = acc(logits, D)  # of a logit
    # lse is a mean of the logits' errors at most as large as the largest; then the sum of V exponentials
    # (chains of at most 128 + V / 2048 + 64 binary32 additions), the exponentials' own few ulp with
    # arguments rounded at |l| 2^-22, and the rounding of lse
    es = el.max(1).values + (256 + V / 2048) * 2.0 ** -24 + 2.0 ** -21 * (1 + logits.abs().max(1).values)
    assert_close(lse, wlse, es, "lse")
    assert_close(loss, want, 2 * es + 2.0 ** -22 * logits.abs().max(1).values, "loss")
    # p has the relative error of exp(l - lse), with the library's lse
    eg = (el + es[:, None] + 2.0 ** -20 * (1 + logits.abs())) * torch.where(t == ignore, 0.0, DL)[:, None] * \
        (logits - wlse[:, None]).exp() + 2.0 ** -22 * g.abs()
    if dX is not None:
        d = g @ W
        assert_close(dX, d, (1 + U8) * (rounded(g, W) + acc(d, V) + eg @ W.abs()) + U8 * d.abs() + 1e-30, "dX")
    if dW is not None:
        d = g.T @ X
        assert_close(dW, d, (1 + U8) * (rounded(g.T, X) + acc(d, T) + eg.T @ X.abs()) + U8 * d.abs() + 1e-30, "dW")


# a vocabulary of one, below a run of 8, odd, ends inside a tile; one token to many; reductions that
# are split; (40000, 10001) takes four pieces of the vocabulary, the last one odd
SIZES = [(1, 1, 8), (1, 7, 64), (1, 50001, 512), (2, 300, 72), (127, 257, 128), (130, 4099, 512), (256, 1024, 256),
         (300, 1000, 1000), (513, 2049, 40), (1100, 3001, 136), (40000, 10001, 64), (3, 8193, 2048)]


@pytest.mark.parametrize("T, V, D", SIZES)
def test_forward_and_backward(T, V, D):
    x, w, t, dloss = _inputs(T, V, D)
    loss, lse = _forward(x, w, t)
    dX, dW = _backward(x, w, t, lse, dloss)
    assert fg.sync_status() == 0
    _check(x, w, t, dloss, loss, lse, dX, dW)


@pytest.mark.parametrize("spread", [30.0, 200.0])
def test_large_logits(spread):
    """Logits of hundreds: their exponentials leave binary32 without the maximum taken out."""
    x, w, t, dloss = _inputs(200, 1500, 256, seed=1, spread=spread)
    loss, lse = _forward(x, w, t)
    dX, dW = _backward(x, w, t, lse, dloss)
    assert fg.sync_status() == 0
    _check(x, w, t, dloss, loss, lse, dX, dW)


def test_equal_dloss_is_not_rounded():
    """The mean over tokens: dloss is one number, here one that bfloat16 rounds by nearly 2^-8.  Each row of
    dW of a target that occurs once is -dloss (1 - p) x_t: to within its own rounding, not dloss's too."""
    T, V, D = 64, 4096, 128
    x, w, t, _ = _inputs(T, V, D, ignored=0.0)
    t = torch.randperm(V, generator=torch.Generator().manual_seed(3))[:T].cuda()
    dloss = torch.full((T,), (1 + 2.0 ** -8 * 0.98) / 64, device="cuda")
    loss, lse = _forward(x, w, t)
    dX, dW = _backward(x, w, t, lse, dloss)
    torch.cuda.synchronize()
    _, _, g, _ = ref.loss_and_gradient(x.to(F64), w.to(F64), t, dloss.to(F64), IGNORE)
    d = (g.T @ x.to(F64))[t]
    rel = (dW[t].to(F64) - d).norm() / d.norm()
    # the result's rounding (rms 2^-8 / sqrt 3 / 1.4) and p - 1's, 2^-9 at most each, but not 2^-8 more
    assert rel < 0.8 * U8


def test_ignored_tokens():
    x, w, t, dloss = _inputs(300, 777, 128, seed=2)
    t[:] = IGNORE  # nothing left
    loss, lse = _forward(x, w, t)
    dX, dW = _backward(x, w, t, lse, dloss)
    assert fg.sync_status() == 0
    assert not loss.any() and not dX.any() and not dW.any() and torch.isfinite(lse).all()
    # an ignored index inside the vocabulary, and an ignored token whose lse and dloss are not finite
    t = torch.randint(777, (300,), generator=torch.Generator().manual_seed(4)).cuda()
    t[:50] = 5
    loss, lse = _forward(x, w, t, ignore=5)
    bad, dl = lse.clone(), dloss.clone()
    bad[:25], dl[:25], bad[25:50] = float("nan"), float("inf"), float("-inf")
    dX, dW = _backward(x, w, t, bad, dl, ignore=5)
    assert fg.sync_status() == 0
    assert not loss[:50].any() and not dX[:50].any()
    ok = torch.where(torch.isfinite(dl), dl, 0)
    _check(x, w, t, ok, loss, lse, dX, dW, ignore=5)


def test_targets_outside_the_vocabulary_are_nan():
    x, w, t, dloss = _inputs(40, 300, 64, ignored=0.0)
    t[3], t[7] = 300, -1
    loss, lse = _forward(x, w, t)
    dX, _ = _backward(x, w, t, lse, dloss)
    assert fg.sync_status() == 0
    at = torch.zeros(40, dtype=torch.bool, device="cuda")
    at[3] = at[7] = True
    assert torch.equal(torch.isnan(loss), at) and torch.equal(torch.isnan(dX).all(1), at)
    assert torch.equal(torch.isnan(dX).any(1), at)


def test_a_row_of_nan_stays_its_own():
    x, w, t, dloss = _inputs(40, 300, 64, ignored=0.0)
    x[5, 3] = float("nan")
    loss, lse = _forward(x, w, t)
    dX, _ = _backward(x, w, t, lse, dloss, dw=False)
    torch.cuda.synchronize()
    assert torch.isnan(loss[5]) and torch.isnan(lse[5]) and torch.isnan(dX[5]).all()
    keep = torch.arange(40, device="cuda") != 5
    assert torch.isfinite(loss[keep]).all() and torch.isfinite(dX[keep]).all()


def test_either_gradient_alone_and_twice_the_same_bits():
    x, w, t, dloss = _inputs(3, 8193, 2048, seed=5)
    loss, lse = _forward(x, w, t)
    a, b = _backward(x, w, t, lse, dloss), _backward(x, w, t, lse, dloss)
    dX, none = _backward(x, w, t, lse, dloss, dw=False)
    _, dW = _backward(x, w, t, lse, dloss, dx=False)
    assert fg.sync_status() == 0
    assert none is None and all(torch.equal(p, q) for p, q in zip(a, b))
    _check(x, w, t, dloss, loss, lse, dX, dW)
    assert all(torch.equal(p, q) for p, q in zip(_forward(x, w, t), (loss, lse)))


def test_gradient_against_differences():
    """Differences of the library's own loss, which is binary32, along the gradients' directions."""
    T, V, D = 100, 999, 256
    x, w, t, _ = _inputs(T, V, D, seed=6, ignored=0.1)
    dloss = torch.full((T,), 1.0 / T, device="cuda")
    loss, lse = _forward(x, w, t)
    dX, dW = _backward(x, w, t, lse, dloss)
    for name, grad in (("x", dX), ("w", dW)):
        base = x if name == "x" else w
        e = grad.to(F64)
        e = e / e.norm() * base.to(F64).norm() * 0.01
        hi, lo = (base.to(F64) + e).bfloat16(), (base.to(F64) - e).bfloat16()
        out = [_forward(v, w, t)[0] if name == "x" else _forward(x, v, t)[0] for v in (hi, lo)]
        slope = ((out[0].to(F64) - out[1].to(F64)) / T).sum()
        want = (grad.to(F64) * (hi.to(F64) - lo.to(F64))).sum()
        # the rounding of the argument is part of the step; the gradient's own rounding, 2^-8 of each of
        # its values, and the curvature over a step of 1 %
        assert abs(slope - want) <= (2 * U8 + 5e-3) * abs(want), (name, float(slope), float(want))


@pytest.mark.parametrize("T, V, D", [(127, 257, 128), (2, 300, 72), (1, 7, 64)])
def test_nothing_outside_is_written(T, V, D):
    x, w, t, dloss = _inputs(T, V, D, seed=7)
    tail = 512
    bufs = [torch.full((n + tail,), 5.0, dtype=torch.bfloat16, device="cuda") for n in (T * D, V * D)]
    red = [torch.full((T + tail,), 5.0, device="cuda") for _ in range(2)]
    fg.linear_cross_entropy(x, w, t, red[0][:T], red[1][:T])
    fg.linear_cross_entropy_backward(x, w, t, red[1][:T], dloss, bufs[0][:T * D].view(T, D), bufs[1][:V * D].view(V, D))
    assert fg.sync_status() == 0
    assert all((b[-tail:] == 5).all() for b in bufs + red)


def test_streams_and_no_tokens():
    x, w, t, dloss = _inputs(200, 1000, 128, seed=8)
    loss, lse = _forward(x, w, t)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = _forward(x, w, t)
    b = _forward(x, w, t, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(p, loss) and torch.equal(q, lse) for p, q in (a, b))
    _forward(x[:0], w, t[:0])
    _, dW = _backward(x[:0], w, t[:0], lse[:0], dloss[:0])
    assert fg.sync_status() == 0
    assert not dW.any()


@pytest.mark.parametrize("state", ["fp32", "bf16", "int8"])
@pytest.mark.parametrize("T, V, D", [(300, 1001, 128), (40000, 10001, 64), (0, 1001, 64)])
def test_step(T, V, D, state):
    """The fused step piece by piece: the first AdamW moment is (1 - beta1) dW in every piece's rows, and
    each weight moves by lr against its gradient's sign."""
    x, w, t, dloss = _inputs(T, V, D, seed=9)
    dloss = dloss * 100
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8}[state]
    W = w.clone()
    m, v = (torch.zeros(V, D, dtype=dt, device="cuda") for _ in range(2))
    q = torch.zeros(2 * V * D // 64, device="cuda") if state == "int8" else None
    loss, lse = _forward(x, w, t)
    dX = torch.full_like(x, float("nan"))
    fg.linear_cross_entropy_step(x, W, t, lse, dloss, dX, m, v, q, opt="adamw", hp=Hparams(lr=1e-2, weight_decay=0.0),
                                 step=1, seed=3)
    assert fg.sync_status() == 0
    if T == 0:
        assert torch.equal(W, w)
        return
    _check(x, w, t, dloss, loss, lse, dX, None)
    X = x.to(F64)
    _, _, g, logits = ref.loss_and_gradient(X, w.to(F64), t, dloss.to(F64), IGNORE)
    d = g.T @ X
    e = 2.0 ** -12 * (g.abs().T @ X.abs())  # of p: the logits' and lse's errors are below 2^-14 here
    # g is rounded with dloss in it, so a target's entries share their rounding: U8, not its deviations
    hot = torch.zeros(V, dtype=torch.bool, device="cuda")
    hot[t[t != IGNORE]] = True
    tol = rounded(g.T, X) + acc(d, T) + e + torch.where(hot[:, None], U8 * d.abs(), 0.0)
    if state == "int8":
        scale = q[:V * D // 64].view(V, -1).repeat_interleave(64, 1).to(F64)
        got, more = m.to(F64) * scale, 0.5 * scale
    else:
        got, more = m.to(F64), (2.0 ** -7 * 0.1 * d.abs() if state == "bf16" else 0.0)
    assert_close(got / 0.1, d, tol * 1.02 + 2.0 ** -22 * d.abs() + more / 0.1 + 1e-12, "m")
    sure = d.abs() > 4 * tol + 1e-4
    moved = (W.to(F64) - w.to(F64) + 1e-2 * d.sign())[sure]
    assert (moved.abs() <= 2.0 ** -7 * (w.to(F64).abs()[sure] + 1e-2) + 1e-4).all()


def test_a_wait_that_runs_out_is_reported():
    x, w, t, dloss = _inputs(600, 9000, 128, seed=10)
    good = _forward(x, w, t)
    torch.cuda.synchronize()
    fg.set_wait_limit_ns(20_000_000)
    try:
        fg.debug_withhold_next_stage()
        _forward(x, w, t)
        assert fg.sync_status() == 6
        fg.debug_withhold_next_stage()
        _backward(x, w, t, good[1], dloss)
        assert fg.sync_status() == 6
    finally:
        fg.set_wait_limit_ns(2_000_000_000)
    again = _forward(x, w, t)
    assert fg.sync_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(again, good))


def test_refusals():
    x, w, t, dloss = _inputs(16, 100, 64)
    loss, lse = torch.empty(16, device="cuda"), torch.empty(16, device="cuda")
    with pytest.raises(TypeError):
        fg.linear_cross_entropy(x, w, t.int(), loss, lse)
    with pytest.raises(TypeError):
        fg.linear_cross_entropy(x, w.float(), t, loss, lse)
    with pytest.raises(TypeError):
        fg.linear_cross_entropy(x, w, t, loss.bfloat16(), lse)
    with pytest.raises(ValueError):
        fg.linear_cross_entropy(x, w, t[:8], loss, lse)
    with pytest.raises(ValueError):
        fg.linear_cross_entropy(x, w[:, ::2], t, loss, lse)
    with pytest.raises(ValueError):
        fg.linear_cross_entropy(x.cpu(), w, t, loss, lse)
    for call in (lambda: fg.linear_cross_entropy(*_inputs(16, 100, 60)[:3], loss, lse),  # 60 is no multiple of 8
                 lambda: fg.linear_cross_entropy(x, w[:0], t, loss, lse),                # no vocabulary
                 lambda: fg.linear_cross_entropy_backward(x, w, t, lse, dloss, None, None)):
        with pytest.raises(fg.ForgeError) as e:
            call()
        assert e.value.status == 1
    assert fg.sync_status() == 0
