"""The head's backward pass with the fused step: as exact as the one that returns dW (needs a GB300)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import operators_reference as ref
from tests.operators_reference import F64, U8
from workloads import Hparams, default_hparams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


# vocabularies whose fused step takes 128 x 64, 128 x 128 and 128 x 256 tiles and pairs; (40000, 10001) several pieces
@pytest.mark.parametrize("T, V, D", [(64, 4096, 128), (64, 1024, 1536), (64, 2432, 1024), (64, 2688, 1024), (64, 8192, 2048),
                                     (2000, 4096, 128), (40000, 10001, 64)])
@pytest.mark.parametrize("state", ["fp32", "bf16", "int8"])
def test_equal_dloss_is_not_rounded(T, V, D, state):
    """The mean over tokens: dloss is one number, here one that bfloat16 rounds by nearly 2^-8.  dX of each token and
    the moment's rows of targets that occur once are off by their own roundings, not by dloss's too."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=gen, device="cuda") / D ** 0.5).bfloat16()
    t = torch.randperm(V, generator=gen, device="cuda")[:T] if T <= V else torch.randint(V, (T,), generator=gen, device="cuda")
    dloss = torch.full((T,), (1 + 2.0 ** -8 * 0.98) / 64, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fg.linear_cross_entropy(x, w, t, loss, lse)
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8}[state]
    W, dX = w.clone(), torch.empty_like(x)
    m, v = (torch.zeros(V, D, dtype=dt, device="cuda") for _ in range(2))
    q = torch.zeros(2 * V * D // 64, device="cuda") if state == "int8" else None
    fg.linear_cross_entropy_step(x, W, t, lse, dloss, dX, m, v, q, hp=Hparams(lr=1e-2, weight_decay=0.0), step=1)
    assert fg.sync_status() == 0
    _, _, g, _ = ref.loss_and_gradient(x.to(F64), w.to(F64), t, dloss.to(F64), -100)

    def off(got, want):
        return float((got - want).norm() / want.norm())

    # The rounding of dX (root mean square below 2^-8 / sqrt 3 / 1.4) and g's, 2^-9 at most each where p is small;
    # dloss's own would add 0.98 * 2^-8 to every entry's error.
    assert off(dX.to(F64), g @ w.to(F64)) < 0.8 * U8
    if state == "int8":
        scale = q[:V * D // 64].view(V, -1).repeat_interleave(64, 1).to(F64)
        got = m.to(F64) * scale
        more = 0.5 / 127 * 4  # half a code of the block's largest, which is below four deviations
    else:
        got, more = m.to(F64), {"fp32": 0.0, "bf16": 2.0 ** -7 / 3 ** 0.5}[state]  # either neighbour: rms below that
    once = t[torch.bincount(t, minlength=V)[t] == 1]
    # the moment is 0.1 of the gradient; what the state's format adds is independent of the rest
    assert off(got[once] / 0.1, (g.T @ x.to(F64))[once]) < ((0.8 * U8) ** 2 + more ** 2) ** 0.5


@pytest.mark.parametrize("opt, state", [(o, s) for o in ("adamw", "nadam", "radam", "lion", "rmsprop", "adagrad", "sgd_momentum")
                                        for s in ("fp32", "bf16", "int8")] + [("sgd", "fp32")])
def test_every_optimizer_takes_the_gradient_itself(opt, state):
    """The step's moments against opt_step on the other form's dW: a factor left out would be one of 500."""
    T, V, D = 500, 1000, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, D, generator=gen, device="cuda").bfloat16()
    w = (torch.randn(V, D, generator=gen, device="cuda") / D ** 0.5).bfloat16()
    t = torch.randint(V, (T,), generator=gen, device="cuda")
    dloss = torch.full((T,), 1 / T, device="cuda")
    loss, lse = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    fg.linear_cross_entropy(x, w, t, loss, lse)
    dX, dW = torch.empty_like(x), torch.empty_like(w)
    fg.linear_cross_entropy_backward(x, w, t, lse, dloss, dX, dW)
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16, "int8": torch.int8}[state]
    use_m, use_v = opt not in ("rmsprop", "adagrad", "sgd"), opt not in ("lion", "sgd_momentum", "sgd")
    runs = []
    for fused in (True, False):
        W = w.clone()
        m, v = (torch.zeros(V, D, dtype=dt, device="cuda") if u else None for u in (use_m, use_v))
        q = torch.zeros(2 * V * D // 64, device="cuda") if state == "int8" else None
        hp = default_hparams(opt, lr=1e-2)
        if fused:
            fg.linear_cross_entropy_step(x, W, t, lse, dloss, None, m, v, q, opt=opt, hp=hp, step=1, seed=5)
        else:
            fg.opt_step(dW.float(), W, m, v, q, opt, hp, 1, 5)
        assert fg.sync_status() == 0
        scale = None if q is None else q.view(2, V, -1).repeat_interleave(64, 2).to(F64)
        runs.append([W.to(F64) - w.to(F64)] + [a.to(F64) if q is None else a.to(F64) * scale[i]
                                               for i, a in enumerate((m, v)) if a is not None])
    # dW's rounding to bf16 and g's (2^-8 each at most; twice that in squares), the moments' to bf16 (either neighbour,
    # 2^-7) and to codes (half of 1/127 of a block's largest, which is below 16 root mean squares of skewed squares)
    tol = 4 * U8 + {"fp32": 0.0, "bf16": 2.0 ** -7, "int8": 0.5 / 127 * 16}[state]
    for i, (a, b) in enumerate(zip(*runs)):
        if i == 0 and opt != "sgd":
            continue  # weights follow their gradient's sign at the first step, and show no factor
        # sgd: the weights' own rounding to either neighbour is in both
        more = 0.0 if i else 2 * float((2.0 ** -7 * w.to(F64)).norm() / b.norm())
        assert float((a - b).norm() / b.norm()) < tol + more, (i, float((a - b).norm() / b.norm()))
