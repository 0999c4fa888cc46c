"""The gated feed-forward block on the GPU against its formulas in binary64 (operators_reference.py)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import operators_reference as ref
from tests.operators_reference import F64, U8, acc, assert_close, rounded
from workloads import Hparams

pytestmark = pytest.mark.gpu

FAST = 2.0 ** -18  # the hardware's exponential and division: a few ulp of binary32, with room


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _empty(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


def _inputs(T, D, F, seed=0, spread=1.0):
    gen = torch.Generator().manual_seed(seed)

    def t(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).bfloat16().cuda()

    w = spread / D ** 0.5
    return {"X": t(T, D), "Wg": t(F, D, std=w), "Wu": t(F, D, std=w), "Wd": t(D, F, std=F ** -0.5), "R": t(T, D),
            "dY": t(T, D, std=0.01), "G": t(T, F, std=spread), "U": t(T, F, std=spread)}


# tokens: 1, below/at/above a tile of 128 and of 256, many; widths that end inside a tile, no multiple
# of 16, the smallest; long reductions that are split; more tiles than the GPU has SMs
SIZES = [(1, 8, 8), (1, 2048, 4096), (2, 64, 520), (17, 72, 200), (127, 256, 512), (129, 1000, 2008), (256, 256, 512),
         (300, 136, 24), (300, 24, 4104), (513, 1024, 776), (1024, 512, 2816), (2100, 640, 1288), (1, 5120, 128)]


def _forward(i, act, save=True, residual=True, stream=None):
    T, D = i["X"].shape
    F = i["Wg"].shape[0]
    Y, G, U = _empty(T, D), *((_empty(T, F), _empty(T, F)) if save else (None, None))
    fg.gated_mlp(i["X"], i["Wg"], i["Wu"], i["Wd"], Y, G, U, residual=i["R"] if residual else None, act=act,
                 stream=stream)
    return Y, G, U


def _check_forward(i, act, Y, G, U, residual):
    d = {k: v.to(F64) for k, v in i.items()}
    D, F = d["X"].shape[1], d["Wg"].shape[0]
    g, u = d["X"] @ d["Wg"].T, d["X"] @ d["Wu"].T
    eg, eu = acc(g, D), acc(u, D)
    if G is not None:
        assert_close(G, g, U8 * g.abs() + (1 + U8) * eg, "G")
        assert_close(U, u, U8 * u.abs() + (1 + U8) * eu, "U")
    a, s = ref.act_both(g, act)
    H = a * u
    # H's own error before its rounding: act has slopes below 1.2
    eh = 1.2 * eg * (u.abs() + eu) + eu * a.abs() + FAST * (H.abs() + g.abs() * u.abs())
    y = H @ d["Wd"].T
    tol = rounded(H, d["Wd"].T) + (1 + U8) * (eh @ d["Wd"].T.abs()) + acc(y, F)
    if residual:
        y = y + d["R"]
    assert_close(Y, y, (1 + U8) * tol + U8 * y.abs(), "Y")


@pytest.mark.parametrize("T, D, F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_forward(T, D, F, act):
    i = _inputs(T, D, F)
    Y, G, U = _forward(i, act)
    assert fg.sync_status() == 0
    _check_forward(i, act, Y, G, U, True)
    Y2, _, _ = _forward(i, act, save=False, residual=False)
    assert fg.sync_status() == 0
    _check_forward(i, act, Y2, None, None, False)


def _backward(i, act, dx=True):
    T, D = i["X"].shape
    F = i["Wg"].shape[0]
    out = _empty(T, D) if dx else None, _empty(F, D), _empty(F, D), _empty(D, F)
    fg.gated_mlp_backward(i["dY"], i["X"], i["G"], i["U"], i["Wg"], i["Wu"], i["Wd"], *out, act=act)
    return out


def _gradients(i, act):
    """(dX, dWg, dWu, dWd) in binary64 and their tolerances before the last rounding."""
    d = {k: v.to(F64) for k, v in i.items()}
    T, D = d["X"].shape
    F = d["Wg"].shape[0]
    a, s = ref.act_both(d["G"], act)
    dH = d["dY"] @ d["Wd"]
    eh = acc(dH, D)
    dG, dU, H = dH * d["U"] * s, dH * a, a * d["U"]
    # what the tensor core's sum and the fast exponential leave of dG, dU and H before their rounding
    eG = eh * (d["U"] * s).abs() + FAST * (dH * d["U"]).abs() * (1 + d["G"].abs())
    eU = eh * a.abs() + FAST * (dH * d["G"]).abs()
    eH = FAST * (d["G"] * d["U"]).abs()
    dX = dG @ d["Wg"] + dU @ d["Wu"]
    tX = (rounded(dG, d["Wg"]).square() + rounded(dU, d["Wu"]).square()).sqrt() + acc(dX, 2 * F) + \
        (1 + U8) * (eG @ d["Wg"].abs() + eU @ d["Wu"].abs())
    want, tol = [dX], [tX]
    for g, e in ((dG, eG), (dU, eU)):
        w = g.T @ d["X"]
        want.append(w)
        tol.append(rounded(g.T, d["X"]) + acc(w, T) + (1 + U8) * (e.T @ d["X"].abs()))
    w = d["dY"].T @ H
    want.append(w)
    tol.append(rounded(d["dY"].T, H) + acc(w, T) + (1 + U8) * (d["dY"].T.abs() @ eH))
    return want, tol


@pytest.mark.parametrize("T, D, F", SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_backward(T, D, F, act):
    i = _inputs(T, D, F, seed=1)
    got = _backward(i, act)
    assert fg.sync_status() == 0
    for g, w, t, name in zip(got, *_gradients(i, act), ("dX", "dWg", "dWu", "dWd")):
        assert_close(g, w, (1 + U8) * t + U8 * w.abs(), name)


# sizes whose products take each tile shape, whole and cut into parts: pairs cut (256 x 4096/14336 down), single
# CTAs on 128 columns with a cut last wave (128 tokens up) and cut (down), on 64 columns cut many times
@pytest.mark.parametrize("T, D, F", [(256, 4096, 14336), (128, 4096, 14336), (19, 184, 6440), (300, 1000, 4000)])
def test_forward_in_every_tile_shape(T, D, F):
    i = _inputs(T, D, F, seed=11)
    Y, G, U = _forward(i, "silu")
    assert fg.sync_status() == 0
    _check_forward(i, "silu", Y, G, U, True)


# pairs whole and cut (1024/2816 and 240 wide), 128 columns cut, 64 columns cut
@pytest.mark.parametrize("T, D, F", [(1024, 1024, 2816), (2683, 2552, 240), (64, 1024, 2816), (128, 512, 1024),
                                     (5, 2256, 1096)])
def test_backward_in_every_tile_shape(T, D, F):
    i = _inputs(T, D, F, seed=12)
    got = _backward(i, "gelu_tanh")
    assert fg.sync_status() == 0
    for g, w, t, name in zip(got, *_gradients(i, "gelu_tanh"), ("dX", "dWg", "dWu", "dWd")):
        assert_close(g, w, (1 + U8) * t + U8 * w.abs(), name)


def test_backward_without_dx_and_twice_the_same_bits():
    i = _inputs(300, 24, 4104, seed=2)  # dX's long reduction is split over several CTAs
    a, b, c = _backward(i, "silu"), _backward(i, "silu"), _backward(i, "silu", dx=False)
    assert fg.sync_status() == 0
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    assert c[0] is None
    for g, w, t, name in zip(c[1:], *(v[1:] for v in _gradients(i, "silu")), ("dWg", "dWu", "dWd")):
        assert_close(g, w, (1 + U8) * t + U8 * w.abs(), name)
    f = [_forward(i, "silu") for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(*f))


def test_gradient_against_differences():
    """d/dX and d/dWd of sum(Y C) by differences of the library's own forward: Y in bf16 limits the
    digits, so the step is large and the direction random; relative error of a directional slope."""
    T, D, F = 64, 256, 512
    i = _inputs(T, D, F, seed=3)
    Y, i["G"], i["U"] = _forward(i, "silu")
    i["dY"] = (torch.randn(T, D, generator=torch.Generator().manual_seed(8)) * 0.01).bfloat16().cuda()
    dX, dWg, dWu, dWd = _backward(i, "silu")
    gen = torch.Generator().manual_seed(4)
    for name, grad in (("X", dX), ("Wg", dWg), ("Wu", dWu), ("Wd", dWd)):
        # along the gradient's own direction, where the slope is the gradient's norm
        e = grad.to(F64)
        e = e / e.norm() * i[name].to(F64).norm() * 0.05
        hi, lo = dict(i), dict(i)
        hi[name], lo[name] = (i[name].to(F64) + e).bfloat16(), (i[name].to(F64) - e).bfloat16()
        step = (hi[name].to(F64) - lo[name].to(F64))
        out = [(_forward(j, "silu", save=False)[0].to(F64) * i["dY"].to(F64)).sum() for j in (hi, lo)]
        slope, want = out[0] - out[1], (grad.to(F64) * step).sum()
        # Y's rounding: T D independent errors below 2^-8 |Y|, in both forwards (seven deviations, H's
        # rounding of the same size within); curvature: the step is 5 % of the argument, whose third-order
        # term is at most a few parts in a thousand of the slope
        noise = 8 * U8 * (Y.to(F64) * i["dY"].to(F64)).square().sum().sqrt() * 2 ** 0.5
        assert abs(slope - want) <= noise + 0.02 * abs(want), (name, float(slope), float(want))


def test_extreme_gates():
    """Gates far out saturate: act(g) is g or 0, no NaN from the exponential; NaN and infinite inputs show
    in their own row alone."""
    T, D, F = 5, 64, 128
    i = _inputs(T, D, F, seed=5)
    i["G"][0], i["G"][1] = 300.0, -300.0
    i["G"][2] = 0.0
    for act in ("silu", "gelu_tanh", "relu"):
        got = _backward(i, act)
        assert fg.sync_status() == 0
        for g, w, t, name in zip(got, *_gradients(i, act), ("dX", "dWg", "dWu", "dWd")):
            assert_close(g, w, (1 + U8) * t + U8 * w.abs() + 1e-30, name)
        j = dict(i, X=i["X"].clone())
        j["X"][3, 2], j["X"][4, 0] = float("nan"), float("inf")
        Y, _, _ = _forward(j, act)
        torch.cuda.synchronize()
        assert torch.isfinite(Y[:3]).all() and not torch.isfinite(Y[3]).any()


@pytest.mark.parametrize("T, D, F", [(17, 72, 200), (129, 1000, 2008), (300, 136, 24)])
def test_nothing_outside_is_written(T, D, F):
    i = _inputs(T, D, F, seed=6)
    tail = 512

    def guarded(*shape):
        n = shape[0] * shape[1]
        b = torch.full((n + tail,), 5.0, dtype=torch.bfloat16, device="cuda")
        return b, b[:n].view(shape)

    bufs = [guarded(T, D), guarded(T, F), guarded(T, F), guarded(T, D), guarded(F, D), guarded(F, D), guarded(D, F)]
    (Y, G, U, dX, dWg, dWu, dWd) = (v for _, v in bufs)
    fg.gated_mlp(i["X"], i["Wg"], i["Wu"], i["Wd"], Y, G, U, residual=i["R"])
    fg.gated_mlp_backward(i["dY"], i["X"], i["G"], i["U"], i["Wg"], i["Wu"], i["Wd"], dX, dWg, dWu, dWd)
    assert fg.sync_status() == 0
    assert all((b[-tail:] == 5).all() for b, _ in bufs)


def test_residual_in_place_streams_and_no_tokens():
    i = _inputs(200, 256, 512, seed=7)
    Y, G, U = _forward(i, "silu")
    r = i["R"].clone()
    fg.gated_mlp(i["X"], i["Wg"], i["Wu"], i["Wd"], r, residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    Y2, G2, U2 = _forward(i, "silu", stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(r, Y) and torch.equal(Y2, Y) and torch.equal(G2, G) and torch.equal(U2, U)
    e = {k: (v[:0] if k in ("X", "R", "dY", "G", "U") else v) for k, v in i.items()}
    _forward(e, "silu")
    out = _backward(e, "silu")
    assert fg.sync_status() == 0
    assert all(not o.any() for o in out[1:])


@pytest.mark.parametrize("state", ["fp32", "bf16", "int8"])
@pytest.mark.parametrize("T", [0, 300])
def test_backward_step(T, state):
    """The fused step behind the block's backward: dX from the old weights, and each weight's first AdamW
    moment is (1 - beta1) dW, which the moments show; the weights move by lr against its sign."""
    D, F, act = 256, 576, "silu"
    i = _inputs(T, D, F, seed=9)
    hp = Hparams(lr=1e-2, weight_decay=0.0)
    layers, old = [], []
    for n, w in enumerate(("Wg", "Wu", "Wd")):
        W = i[w].clone()
        dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8}[state]
        m, v = (torch.zeros(W.shape, dtype=dt, device="cuda") for _ in range(2))
        q = torch.zeros(2 * W.numel() // 64, device="cuda") if state == "int8" else None
        layers.append((W, m, v, q, 11 + n))
        old.append(W.clone())
    dX = _empty(T, D)
    fg.gated_mlp_backward_step(i["dY"], i["X"], i["G"], i["U"], *layers, dX, act=act, opt="adamw", hp=hp, step=1)
    assert fg.sync_status() == 0
    if T == 0:
        assert all(torch.equal(W, o) for (W, *_), o in zip(layers, old))
        return
    want, tol = _gradients(i, act)
    assert_close(dX, want[0], (1 + U8) * tol[0] + U8 * want[0].abs(), "dX")
    for (W, m, v, q, _), w, t, o, name in zip(layers, want[1:], tol[1:], old, ("Wg", "Wu", "Wd")):
        if state == "int8":
            scale = q[:W.numel() // 64].view(W.shape[0], -1).repeat_interleave(64, 1).to(F64)
            got, more = m.to(F64) * scale, 0.5 * scale
        else:
            # bf16 moments are rounded to either neighbour, at most 2^-7 away
            got, more = m.to(F64), (2.0 ** -7 * 0.1 * w.abs() if state == "bf16" else 0.0)
        assert_close(got / 0.1, w, t * 1.02 + 2.0 ** -22 * w.abs() + more / 0.1 + 1e-12, f"m of {name}")
        # the first AdamW step moves every weight by lr against its gradient's sign, up to eps; the weight
        # is then rounded to either neighbour, at most 2^-7 away
        sure = w.abs() > 4 * t + 1e-5
        moved = (W.to(F64) - o.to(F64) + 1e-2 * w.sign())[sure]
        assert (moved.abs() <= 2.0 ** -7 * (o.to(F64).abs()[sure] + 1e-2) + 1e-4).all(), name


def test_a_wait_that_runs_out_is_reported():
    i = _inputs(300, 256, 512, seed=10)
    good = _forward(i, "silu")
    torch.cuda.synchronize()
    fg.set_wait_limit_ns(20_000_000)
    try:
        for call in (lambda: _forward(i, "silu"), lambda: _backward(i, "silu")):
            fg.debug_withhold_next_stage()
            call()
            assert fg.sync_status() == 6
    finally:
        fg.set_wait_limit_ns(2_000_000_000)
    again = _forward(i, "silu")
    assert fg.sync_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(again, good))


def test_refusals():
    i = _inputs(16, 64, 128)
    Y, G, U = _empty(16, 64), _empty(16, 128), _empty(16, 128)
    args = (i["X"], i["Wg"], i["Wu"], i["Wd"])
    with pytest.raises(TypeError):
        fg.gated_mlp(i["X"].float(), *args[1:], Y)
    with pytest.raises(ValueError):
        fg.gated_mlp(*args, Y[:8])
    with pytest.raises(ValueError):
        fg.gated_mlp(i["X"], i["Wg"], i["Wu"][:64], i["Wd"], Y)
    with pytest.raises(ValueError):
        fg.gated_mlp(*args, Y, act="tanh")
    with pytest.raises(ValueError):
        fg.gated_mlp(i["X"], i["Wg"], i["Wu"], i["Wd"].t().contiguous().t(), Y)  # not row-major
    with pytest.raises(ValueError):
        fg.gated_mlp(*(t.cpu() for t in args), Y)
    odd = _inputs(16, 60, 128)
    for call, status in (
            (lambda: fg.gated_mlp(*args, Y, G), 1),  # G without U
            (lambda: fg.gated_mlp(odd["X"], odd["Wg"], odd["Wu"], odd["Wd"], _empty(16, 60)), 1),  # 60 is no multiple of 8
            (lambda: fg.gated_mlp(_empty(17 * 64)[8:8 + 16 * 64].view(16, 64), *args[1:], Y), 3)):  # 16-byte aligned only
        with pytest.raises(fg.ForgeError) as e:
            call()
        assert e.value.status == status
    with pytest.raises(TypeError):
        f, b = torch.zeros(128, 64, device="cuda"), torch.zeros(128, 64, dtype=torch.bfloat16, device="cuda")
        d = torch.zeros(64, 128, device="cuda")
        fg.gated_mlp_backward_step(Y, i["X"], i["G"], i["U"], (i["Wg"], f, f.clone(), None, 0),
                                   (i["Wu"], b, b.clone(), None, 1), (i["Wd"], d, d.clone(), None, 2))
    assert fg.sync_status() == 0
