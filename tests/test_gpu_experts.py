"""Products grouped by expert on the GPU against their formulas in binary64, expert by expert (the tolerances of the
dense products: operators_reference.py)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import operators_reference as ref
from tests import test_gpu_gated as dense
from tests.operators_reference import F64, U8, acc, assert_close
from workloads import Hparams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


FILL = 7.0  # what results hold before a call


def _full(*shape):
    return torch.full(shape, FILL, dtype=torch.bfloat16, device="cuda")


def _offsets(sizes, lead=0):
    return torch.tensor([lead] + sizes).cumsum(0).to(torch.int32).cuda()


def _runs(sizes, lead=0):
    at = lead
    for e, n in enumerate(sizes):
        yield e, slice(at, at + n)
        at += n


def _outside(rows, sizes, lead):
    """Rows of no expert."""
    out = torch.ones(rows, dtype=torch.bool, device="cuda")
    out[lead:lead + sum(sizes)] = False
    return out


def _spread(rng_seed, experts, most):
    gen = torch.Generator().manual_seed(rng_seed)
    return [int(n) for n in torch.randint(0, most + 1, (experts,), generator=gen)]


# runs: none, one row, around tiles of 32, 64, 128 and 256 rows, slices of 64, one large among small ones; lead and
# tail: rows before the first run and behind the last; widths that end inside a tile, no multiple of 64 or 16
CASES = [
    ([1], 0, 0, 8, 8), ([0, 1, 0], 0, 0, 64, 520), ([3, 0, 5, 1], 2, 3, 72, 200), ([2, 2], 0, 0, 2048, 4096),
    ([31, 32, 33, 0, 7], 0, 9, 256, 136), (_spread(1, 64, 20), 1, 5, 512, 264), (_spread(2, 130, 3), 0, 40, 64, 96),
    ([129, 0, 127, 1, 63, 65], 0, 1, 256, 512), ([64, 64, 128], 0, 0, 128, 192), ([300, 17], 5, 0, 136, 24),
    ([333], 0, 0, 1000, 264), ([700, 513, 0, 900], 0, 77, 640, 1288), ([255, 256, 257, 511], 3, 0, 1024, 776),
    ([0, 4000, 1, 0, 30], 0, 2, 512, 320), ([0, 0, 0], 4, 4, 64, 64),
]
# on pairs, where a run's last tile is as wide as its rest: every width, at its edges
CASES += [([32 * k + d for k in range(9) for d in (0, 1, 31)], 0, 3, 136, 328)]
# there, few tiles with a long reduction, which are cut
CASES += [([150, 0, 200], 1, 2, 104, 5000)]
# few tiles of gradients with long runs, which are cut; a run of fewer slices than parts
CASES += [([12000, 0, 70], 1, 2, 72, 136)]


def _tensor(gen, *shape, std=1.0):
    return (torch.randn(*shape, generator=gen) * std).bfloat16().cuda()


def _gated_inputs(sizes, lead, tail, D, F, seed=0):
    gen = torch.Generator().manual_seed(seed)
    R, E, w = lead + sum(sizes) + tail, len(sizes), 1.0 / D ** 0.5
    i = {"X": _tensor(gen, R, D), "Wg": _tensor(gen, E, F, D, std=w), "Wu": _tensor(gen, E, F, D, std=w),
         "Wd": _tensor(gen, E, D, F, std=F ** -0.5), "dY": _tensor(gen, R, D, std=0.01), "G": _tensor(gen, R, F),
         "U": _tensor(gen, R, F)}
    out = _outside(R, sizes, lead)
    for name in ("X", "dY", "G", "U"):  # rows of no expert count for nothing, whatever they hold
        i[name][out] = float("nan")
    return i


def _of(i, e, r):
    """One expert's rows and weights, as the dense block takes them."""
    d = {k: i[k][r] for k in ("X", "dY", "G", "U")}
    return {**d, **{k: i[k][e] for k in ("Wg", "Wu", "Wd")}, "R": torch.zeros_like(d["X"])}


def _forward(i, offsets, act, save=True, stream=None):
    (R, D), F = i["X"].shape, i["Wg"].shape[1]
    Y, G, U = _full(R, D), *((_full(R, F), _full(R, F)) if save else (None, None))
    fg.expert_gated_mlp(i["X"], i["Wg"], i["Wu"], i["Wd"], offsets, Y, G, U, act=act, stream=stream)
    return Y, G, U


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_gated_forward(case, act):
    sizes, lead, tail, D, F = CASES[case]
    i = _gated_inputs(sizes, lead, tail, D, F)
    Y, G, U = _forward(i, _offsets(sizes, lead), act)
    Y2, _, _ = _forward(i, _offsets(sizes, lead), act, save=False)
    assert fg.sync_status() == 0
    assert torch.equal(Y, Y2)
    for e, r in _runs(sizes, lead):
        if r.stop > r.start:
            dense._check_forward(_of(i, e, r), act, Y[r], G[r], U[r], False)
    out = _outside(len(Y), sizes, lead)
    assert all((t[out] == FILL).all() for t in (Y, G, U))


def _backward(i, offsets, act, dx=True):
    (R, D), (E, F, _) = i["X"].shape, i["Wg"].shape
    out = _full(R, D) if dx else None, _full(E, F, D), _full(E, F, D), _full(E, D, F)
    fg.expert_gated_mlp_backward(i["dY"], i["X"], i["G"], i["U"], i["Wg"], i["Wu"], i["Wd"], offsets, *out, act=act)
    return out


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_gated_backward(case, act):
    sizes, lead, tail, D, F = CASES[case]
    i = _gated_inputs(sizes, lead, tail, D, F, seed=1)
    dX, *dW = _backward(i, _offsets(sizes, lead), act)
    none, *dW2 = _backward(i, _offsets(sizes, lead), act, dx=False)
    assert fg.sync_status() == 0
    for e, r in _runs(sizes, lead):
        if r.stop == r.start:
            assert not any(w[e].any() for w in dW)
            continue
        want, tol = dense._gradients(_of(i, e, r), act)
        for got, c, t, name in zip((dX[r], *(w[e] for w in dW)), want, tol, ("dX", "dWg", "dWu", "dWd")):
            assert_close(got, c, (1 + U8) * t + U8 * c.abs(), f"{name} of expert {e}")
    assert (dX[_outside(len(dX), sizes, lead)] == FILL).all()
    assert all(torch.equal(a, b) for a, b in zip(dW, dW2))


@pytest.mark.parametrize("case", range(len(CASES)))
def test_linear(case):
    sizes, lead, tail, D, F = CASES[case]
    gen = torch.Generator().manual_seed(2)
    R, E = lead + sum(sizes) + tail, len(sizes)
    X, dY, W = _tensor(gen, R, D), _tensor(gen, R, F), _tensor(gen, E, F, D, std=D ** -0.5)
    out = _outside(R, sizes, lead)
    X[out], dY[out] = float("nan"), float("inf")
    off = _offsets(sizes, lead)
    Y, dX, dW, dX1, dW1 = _full(R, F), _full(R, D), _full(E, F, D), _full(R, D), _full(E, F, D)
    fg.expert_linear(X, W, off, Y)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    fg.expert_linear_backward(dY, X, W, off, dX1, None)
    fg.expert_linear_backward(dY, X, W, off, None, dW1)
    assert fg.sync_status() == 0
    assert torch.equal(dX, dX1) and torch.equal(dW, dW1)
    for e, r in _runs(sizes, lead):
        if r.stop == r.start:
            assert not dW[e].any()
            continue
        x, d, w = X[r].to(F64), dY[r].to(F64), W[e].to(F64)
        for got, c, k, name in ((Y[r], x @ w.T, D, "Y"), (dX[r], d @ w, F, "dX"), (dW[e], d.T @ x, r.stop - r.start, "dW")):
            assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), f"{name} of expert {e}")
    assert (Y[out] == FILL).all() and (dX[out] == FILL).all()


@pytest.mark.parametrize("sizes", [[70, 1, 33, 200], [300, 290, 310, 280], [5, 0, 9, 2]])
def test_a_neighbour_that_is_not_finite_stays_out(sizes):
    """Runs that end inside a slice of 64 rows: the next expert's infinities and NaN enter no sum of this one."""
    i = _gated_inputs(sizes, 0, 0, 128, 192, seed=3)
    clean = _backward(i, _offsets(sizes), "silu")
    y = _forward(i, _offsets(sizes), "silu")[0]
    bad = list(_runs(sizes))[2][1]
    for name, v in (("X", float("inf")), ("dY", float("nan")), ("G", float("-inf")), ("U", float("nan"))):
        i[name][bad] = v
    for name in ("Wg", "Wu", "Wd"):
        i[name][2] = float("nan")
    dirty = _backward(i, _offsets(sizes), "silu")
    y2 = _forward(i, _offsets(sizes), "silu")[0]
    assert fg.sync_status() == 0
    for e, r in _runs(sizes):
        if e != 2:
            assert torch.equal(dirty[0][r], clean[0][r]) and torch.equal(y2[r], y[r])
            assert all(torch.equal(a[e], b[e]) for a, b in zip(dirty[1:], clean[1:]))


def test_offsets_out_of_order_and_out_of_range():
    """Taken as the nearest ones in order and within the rows."""
    R, E, D, F = 100, 6, 64, 72
    gen = torch.Generator().manual_seed(4)
    X, dY, W = _tensor(gen, R, D), _tensor(gen, R, F), _tensor(gen, E, F, D)
    got, want = [], []
    for given, out in (([-5, 20, 10, 60, 300, 50, 2**31 - 1], got), ([0, 20, 20, 60, 100, 100, 100], want)):
        off = torch.tensor(given).to(torch.int32).cuda()
        Y, dX, dW = _full(R, F), _full(R, D), _full(E, F, D)
        fg.expert_linear(X, W, off, Y)
        fg.expert_linear_backward(dY, X, W, off, dX, dW)
        out += [Y, dX, dW]
    assert fg.sync_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_no_rows():
    X, dY = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
    W, off, dW = _full(3, 72, 64), torch.zeros(4, dtype=torch.int32, device="cuda"), _full(3, 72, 64)
    fg.expert_linear(X, W, off, dY)
    fg.expert_linear_backward(dY, X, W, off, torch.empty_like(X), dW)
    assert fg.sync_status() == 0
    assert not dW.any()
    out = [_full(3, 72, 64), _full(3, 72, 64), _full(3, 64, 72)]
    fg.expert_gated_mlp_backward(X, X, dY, dY, W, W, _full(3, 64, 72), off, None, *out)
    assert fg.sync_status() == 0
    assert not any(t.any() for t in out)


@pytest.mark.parametrize("D, F", [(520, 1032), (512, 1024)])
def test_tensors_that_end_with_their_memory(D, F):
    """Runs shorter than a slice at the very end of an allocation of whole pages: nothing past it is read."""
    sizes = [82, 20, 57, 0, 10, 7, 0, 36, 110, 8, 237, 0, 2, 117, 237, 13]
    R, E = sum(sizes), len(sizes)
    gen = torch.Generator().manual_seed(8)

    def at_the_end(t):
        whole = torch.zeros(22 << 19 << 1, dtype=torch.bfloat16, device="cuda")  # 44 MiB, a segment of its own
        v = whole[-t.numel():].view(t.shape)
        v.copy_(t)
        return v
    X, dY, U = at_the_end(_tensor(gen, R, D)), at_the_end(_tensor(gen, R, D, std=0.01)), at_the_end(_tensor(gen, R, F))
    i = {"X": X, "dY": dY, "G": at_the_end(_tensor(gen, R, F)), "U": U, "Wg": _tensor(gen, E, F, D, std=D ** -0.5),
         "Wu": _tensor(gen, E, F, D, std=D ** -0.5), "Wd": _tensor(gen, E, D, F, std=F ** -0.5)}
    dX, *dW = _backward(i, _offsets(sizes), "silu")
    assert fg.sync_status() == 0
    for e, r in _runs(sizes):
        if r.stop > r.start:
            want, tol = dense._gradients(_of(i, e, r), "silu")
            for got, c, t in zip((dX[r], *(w[e] for w in dW)), want, tol):
                assert_close(got, c, (1 + U8) * t + U8 * c.abs(), f"expert {e}")


def test_gradients_against_differences():
    """Along random directions, in binary64, about the kernel's own inputs: d/dh of sum(C * block(inputs + h direction))."""
    sizes, D, F = [9, 0, 70, 33], 64, 136
    i = _gated_inputs(sizes, 0, 0, D, F, seed=5)
    off, names = _offsets(sizes), ("X", "Wg", "Wu", "Wd")
    C = i["dY"]

    def value(v):
        total = 0.0
        for e, r in _runs(sizes):
            g, u = v["X"][r] @ v["Wg"][e].T, v["X"][r] @ v["Wu"][e].T
            total = total + (C[r].to(F64) * ((ref.act_both(g, "silu")[0] * u) @ v["Wd"][e].T)).sum()
        return total
    v = {n: i[n].to(F64) for n in names}
    # the backward pass starts from G and U as the forward pass left them
    _, i["G"], i["U"] = _forward(i, off, "silu")
    got = dict(zip(names, _backward(i, off, "silu")))
    gen = torch.Generator().manual_seed(6)
    for n in names:
        for e, r in _runs(sizes):
            if r.stop == r.start:
                continue
            at = r if n == "X" else e
            d = torch.zeros_like(v[n])
            d[at] = torch.randn(d[at].shape, generator=gen, dtype=F64).cuda()
            h = 1e-4
            diff = (value({**v, n: v[n] + h * d}) - value({**v, n: v[n] - h * d})) / (2 * h)
            own = (got[n][at].to(F64) * d[at]).sum()
            # a random direction takes the square root of the sum of the elements' squared errors: each at most a few
            # half steps of bf16 (the result, and dG, dU, H, G and U before it) of its own size; seven deviations
            tol = 7 * 4 * U8 * (got[n][at].to(F64) * d[at]).square().sum().sqrt()
            assert abs(diff - own) < tol, (n, e, diff.item(), own.item(), tol.item())
    lin = {n: i[n].to(F64) for n in ("X",)} | {"W": i["Wg"].to(F64)}
    dX, dW = _full(*i["X"].shape), _full(*i["Wg"].shape)
    dZ = i["G"]
    fg.expert_linear_backward(dZ, i["X"], i["Wg"], off, dX, dW)
    for n, g in (("X", dX), ("W", dW)):
        d = torch.randn(g.shape, generator=gen, dtype=F64).cuda()

        def out(x, w):
            return sum((dZ[r].to(F64) * (x[r] @ w[e].T)).sum() for e, r in _runs(sizes))
        args = {"X": lin["X"], "W": lin["W"]}
        up, down = {**args, n: args[n] + 1e-3 * d}, {**args, n: args[n] - 1e-3 * d}
        diff = (out(up["X"], up["W"]) - out(down["X"], down["W"])) / 2e-3
        own, tol = (g.to(F64) * d).sum(), 7 * 2 * U8 * (g.to(F64) * d).square().sum().sqrt()
        assert abs(diff - own) < tol


@pytest.mark.parametrize("experts, rows", [(1024, 1), (1024, 700), (1000, 5000), (1, 4097)])
def test_many_experts_and_one(experts, rows):
    gen = torch.Generator().manual_seed(10)
    D, F = 64, 72
    cuts = torch.randint(0, rows + 1, (experts - 1,), generator=gen).sort().values.tolist()
    sizes = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    X, dY, W = _tensor(gen, rows, D), _tensor(gen, rows, F), _tensor(gen, experts, F, D, std=D ** -0.5)
    off = _offsets(sizes)
    Y, dX, dW = _full(rows, F), _full(rows, D), _full(experts, F, D)
    fg.expert_linear(X, W, off, Y)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    assert fg.sync_status() == 0
    which = torch.repeat_interleave(torch.arange(experts), torch.tensor(sizes)).cuda()
    x, d, w = X.to(F64), dY.to(F64), W.to(F64)
    # binary32 sums of 64 and 72 products: far inside one more half step of bf16
    y = torch.einsum("rd,rfd->rf", x, w[which])
    g = torch.einsum("rf,rfd->rd", d, w[which])
    h = torch.zeros(experts, F, D, dtype=F64, device="cuda")
    for e, r in _runs(sizes):
        if r.stop > r.start:
            h[e] = d[r].T @ x[r]
    for got, c, k, name in ((Y, y, D, "Y"), (dX, g, F, "dX"), (dW, h, rows, "dW")):
        assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), name)


def test_rows_and_weights_past_32_bits():
    """Element numbers over 2^32 in X and dX (rows) and in W and dW (experts): the last rows and the last experts."""
    D, F = 8192, 64
    sizes = [260000, 0, 300000, 5, 40]
    R, E = sum(sizes), len(sizes)
    X = torch.zeros(R, D, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(11)
    tail = _tensor(gen, 45, D)
    X[-45:] = tail
    W, dY = _tensor(gen, E, F, D, std=D ** -0.5), torch.zeros(R, F, dtype=torch.bfloat16, device="cuda")
    dY[-45:] = _tensor(gen, 45, F)
    off = _offsets(sizes)
    Y, dX, dW = _full(R, F), _full(R, D), _full(E, F, D)
    fg.expert_linear(X, W, off, Y)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    assert fg.sync_status() == 0
    assert not Y[:-45].any() and not dX[:-45].any() and not dW[:3].any()
    for e, r in ((3, slice(R - 45, R - 40)), (4, slice(R - 40, R))):
        x, d, w = X[r].to(F64), dY[r].to(F64), W[e].to(F64)
        for got, c, k, name in ((Y[r], x @ w.T, D, "Y"), (dX[r], d @ w, F, "dX"), (dW[e], d.T @ x, 64, "dW")):
            assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), f"{name} of expert {e}")
    del X, dY, Y, dX
    E, D, F = 70, 8192, 8192
    sizes = [0] * E
    sizes[0], sizes[68], sizes[69] = 3, 40, 90
    R = sum(sizes)
    W = torch.zeros(E, F, D, dtype=torch.bfloat16, device="cuda")
    for e in (0, 68, 69):
        W[e] = _tensor(gen, F, D, std=D ** -0.5)
    X, dY, off = _tensor(gen, R, D), _tensor(gen, R, F, std=0.1), _offsets(sizes)
    Y, dX, dW = _full(R, F), _full(R, D), _full(E, F, D)
    fg.expert_linear(X, W, off, Y)
    fg.expert_linear_backward(dY, X, W, off, dX, dW)
    m = torch.zeros(E, F, D, dtype=torch.bfloat16, device="cuda")
    old = W[69].clone()
    fg.expert_linear_backward_step(dY, X, W, off, None, m, None, None, opt="sgd_momentum",
                                   hp=Hparams(lr=1.0, momentum=0.0, weight_decay=0.0), step=1)
    assert fg.sync_status() == 0
    assert not dW[1:68].any() and not m[1:68].any()
    for e, r in _runs(sizes):
        if r.stop == r.start:
            continue
        x, d = X[r].to(F64), dY[r].to(F64)
        w = (old if e == 69 else W[e]).to(F64)
        if e == 69:
            for got, c, k, name in ((Y[r], x @ w.T, D, "Y"), (dX[r], d @ w, F, "dX")):
                assert_close(got, c, U8 * c.abs() + (1 + U8) * acc(c, k), f"{name} of expert {e}")
        c = d.T @ x
        assert_close(dW[e], c, U8 * c.abs() + (1 + U8) * acc(c, 128), f"dW of expert {e}")
        # the moment is the gradient, rounded stochastically: a whole step
        assert_close(m[e], c, 2 * U8 * c.abs() + (1 + 2 * U8) * acc(c, 128), f"m of expert {e}")
