"""The fused step over experts' weights: bit for bit the two-phase update of one matrix that stacks the experts, and the
gated block's gradients against the formulas."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import test_gpu_gated as dense
from tests.operators_reference import U8, assert_close
from tests.test_gpu_experts import _full, _gated_inputs, _of, _offsets, _outside, _runs, _tensor
from workloads import Hparams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


HP = Hparams(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1, momentum=0.9, alpha=0.95, lr_decay=0.01,
             momentum_decay=0.004)
USES = {"adamw": "mv", "nadam": "mv", "radam": "mv", "lion": "m", "rmsprop": "v", "adagrad": "v", "sgd": "", "sgd_momentum": "m"}


def _states(gen, shape, opt, state):
    n = shape[0] * shape[1] * shape[2]
    out = {}
    for name in "mv":
        if name not in USES[opt]:
            out[name] = None
        elif state == "int8":
            out[name] = torch.randint(0 if name == "v" else -127, 128, shape, generator=gen, dtype=torch.int8).cuda()
        else:
            t = torch.randn(shape, generator=gen) * 1e-2
            out[name] = (t.abs() if name == "v" else t).to(torch.float32 if state == "fp32" else torch.bfloat16).cuda()
    q = (torch.rand(2 * n // 64, generator=gen) * 1e-4).cuda() if state == "int8" and USES[opt] else None
    return out["m"], out["v"], q


def _clone(*ts):
    return [None if t is None else t.clone() for t in ts]


# single CTAs (ragged widths; few experts) and CTA pairs (many experts, wide weights); empty runs, single rows, a long one
SHAPES = [([3, 0, 70, 1], 2, 3, 72, 192), ([129, 0, 64, 500], 0, 0, 256, 384), ([5, 0, 130, 2] * 10, 0, 7, 256, 256),
          ([40, 0, 300, 7, 64], 0, 0, 1088, 1024), ([9, 0, 257], 1, 0, 2048, 1536)]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("opt, state", [(o, s) for o in USES for s in ("fp32", "bf16", "int8") if o != "sgd" or s == "fp32"])
def test_linear_step_is_the_stacked_two_phase_step(shape, opt, state):
    sizes, lead, tail, D, F = SHAPES[shape]
    if state == "int8" and D % 64:
        D = 64
    gen = torch.Generator().manual_seed(shape)
    R, E = lead + sum(sizes) + tail, len(sizes)
    X, dY, W = _tensor(gen, R, D), _tensor(gen, R, F, std=0.1), _tensor(gen, E, F, D, std=0.05)
    out = _outside(R, sizes, lead)
    X[out], dY[out] = float("nan"), float("inf")
    m, v, q = _states(gen, (E, F, D), opt, state)
    dW = torch.zeros(E, F, D, device="cuda")
    for e, r in _runs(sizes, lead):
        if r.stop > r.start:
            fg.dw_gemm(dY[r].clone(), X[r].clone(), dW[e])
    want = _clone(W, m, v, q)
    fg.opt_step(dW.view(E * F, D), want[0].view(E * F, D), *(None if t is None else t.view(E * F, D) for t in want[1:3]), want[3],
                opt=opt, hp=HP, step=4, seed=(1 << 60) + 5)
    dX, dX2 = _full(R, D), _full(R, D)
    fg.expert_linear_backward(dY, X, W, _offsets(sizes, lead), dX, None)
    got = _clone(W, m, v, q)
    fg.expert_linear_backward_step(dY, X, got[0], _offsets(sizes, lead), dX2, *got[1:], opt=opt, hp=HP, step=4, seed=(1 << 60) + 5)
    assert fg.sync_status() == 0
    for a, b, name in zip(got, want, ("W", "m", "v", "qscales")):
        assert a is None or torch.equal(a, b), name
    assert torch.equal(dX, dX2)  # from the weights before the step
    got = _clone(W, m, v, q)
    fg.expert_linear_backward_step(dY, X, got[0], _offsets(sizes, lead), None, *got[1:], opt=opt, hp=HP, step=4, seed=(1 << 60) + 5)
    assert fg.sync_status() == 0
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("case", [([3, 0, 5, 1], 2, 3, 72, 200), ([129, 0, 127, 1, 63, 65], 0, 1, 256, 512),
                                  ([300, 0, 17], 0, 0, 640, 1288), ([20, 90, 0, 41] * 10, 0, 0, 256, 512)])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "relu"])
def test_gated_step(case, act):
    """With momentum 0 the FP32 moment is the gradient itself."""
    sizes, lead, tail, D, F = case
    i = _gated_inputs(sizes, lead, tail, D, F, seed=1)
    R, E = i["X"].shape[0], len(sizes)
    hp = Hparams(lr=0.5, momentum=0.0, weight_decay=0.0)
    layers, old = [], {}
    for k, name in enumerate(("Wg", "Wu", "Wd")):
        w = i[name].clone()
        old[name] = i[name]
        layers.append((w, torch.full(w.shape, 3.0, device="cuda"), None, None, k))
    dX, dX2 = _full(R, D), _full(R, D)
    fg.expert_gated_mlp_backward(i["dY"], i["X"], i["G"], i["U"], i["Wg"], i["Wu"], i["Wd"], _offsets(sizes, lead), dX,
                                 *(torch.empty_like(i[n]) for n in ("Wg", "Wu", "Wd")), act=act)
    fg.expert_gated_mlp_backward_step(i["dY"], i["X"], i["G"], i["U"], *layers, _offsets(sizes, lead), dX2, act=act,
                                      opt="sgd_momentum", hp=hp, step=2)
    assert fg.sync_status() == 0
    assert torch.equal(dX, dX2)
    for e, r in _runs(sizes, lead):
        if r.stop == r.start:
            assert not any(m[e].any() for _, m, *_ in layers)
            assert all(torch.equal(w[e], old[n][e]) for (w, *_), n in zip(layers, ("Wg", "Wu", "Wd")))
            continue
        want, tol = dense._gradients(_of(i, e, r), act)
        for (w, m, *_), c, t, name in zip(layers, want[1:], tol[1:], ("Wg", "Wu", "Wd")):
            assert_close(m[e], c, t, f"d{name} of expert {e}")
            new = old[name][e].double() - 0.5 * m[e].double()
            # stochastic rounding: one of the two neighbours, a whole step of bf16 at most (2 U8), and binary32 before it
            assert_close(w[e], new, 2 * U8 * new.abs() + 2.0 ** -23 * old[name][e].double().abs() + 2.0 ** -133, name)


def test_no_rows_is_a_step_with_gradient_zero():
    gen = torch.Generator().manual_seed(3)
    W = _tensor(gen, 3, 72, 64)
    m, v = torch.randn(3, 72, 64, generator=gen).cuda(), torch.rand(3, 72, 64, generator=gen).cuda()
    X, dY, off = (torch.empty(0, n, dtype=torch.bfloat16, device="cuda") for n in (64, 72, 0))
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    want, got = _clone(W, m, v), _clone(W, m, v)
    fg.opt_step(torch.zeros(216, 64, device="cuda"), *(t.view(216, 64) for t in want), None, opt="adamw", hp=HP, step=2, seed=9)
    fg.expert_linear_backward_step(dY, X, got[0], off, None, got[1], got[2], None, opt="adamw", hp=HP, step=2, seed=9)
    # the same where rows belong to no expert
    rows = torch.full((40, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    got2 = _clone(W, m, v)
    fg.expert_linear_backward_step(torch.full((40, 72), float("nan"), dtype=torch.bfloat16, device="cuda"), rows, got2[0], off, None,
                                   got2[1], got2[2], None, opt="adamw", hp=HP, step=2, seed=9)
    assert fg.sync_status() == 0
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(got, want, got2))
