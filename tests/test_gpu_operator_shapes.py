"""Every way in which the operators' products are run -- the few-token kernel's instantiations, tiles of each width
whole, cut along the reduction, and cut in the last wave only -- against the formulas in binary64.  The sizes are
asserted to take the way that they stand for, so that another choice of tiles cannot leave one untested unnoticed
(needs a GB300)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from backward_optimizer_gb300.operators import gated_launch_shape, loss_launch_shape
from tests import test_gpu_gated as gated
from tests import test_gpu_loss as loss
from tests.operators_reference import U8, assert_close
from workloads import Hparams

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


# ------------------------------------------------------------------ one to four tokens
# A row's 16-byte runs are shared by 512 lanes, so the instantiations are by ceil(width / 4096), of d_model for gate and
# up and of d_ff for down: up to 5 for one and two tokens, up to 2 for three and four.  Widths that are no multiple
# of a lane's run times the lanes, outputs that are no multiple of the blocks.
FEW = [(T, D, F) for T in (1, 2) for D, F in ((2048, 5632), (512, 10008), (5120, 13000), (256, 17408), (9000, 64), (14336, 64),
                                              (17000, 72), (4096, 14336), (5120, 17408))] + \
      [(T, D, F) for T in (3, 4) for D, F in ((512, 1408), (4096, 8192), (5120, 4104), (8192, 4000))]


def test_the_sizes_take_every_few_token_kernel():
    runs = lambda k: -(-k // 4096)  # noqa: E731
    for T, most in ((1, 5), (2, 5), (3, 2), (4, 2)):
        assert {runs(D) for t, D, _ in FEW if t == T} == set(range(1, most + 1))
        assert {runs(F) for t, _, F in FEW if t == T} == set(range(1, most + 1))


@pytest.mark.parametrize("T, D, F", FEW)
def test_few_tokens(T, D, F):
    assert gated_launch_shape(T, D, F, "up")["tile_cols"] == gated_launch_shape(T, D, F, "down")["tile_cols"] == 0
    i = gated._inputs(T, D, F, seed=T)
    for save, residual in ((True, True), (False, False)):
        Y, G, U = gated._forward(i, "silu", save=save, residual=residual)
        assert fg.sync_status() == 0
        gated._check_forward(i, "silu", Y, G, U, residual)


# ------------------------------------------------------------------ tiles


def _way(s):
    return s["tile_cols"], "whole" if s["cut"] == 0 else "cut" if s["whole"] == 0 else "tail"


GATED = [((886, 3256, 104), {"up": (64, "cut"), "down": (128, "whole"), "dh": (64, "cut")}),
         ((669, 768, 584), {"up": (64, "whole"), "dh": (64, "whole")}),
         ((6, 9032, 5536), {"up": (128, "whole"), "down": (128, "cut"), "dh": (128, "cut")}),
         ((15, 7888, 2536), {"up": (128, "cut")}),
         ((6, 4992, 10024), {"up": (128, "tail")}),
         ((138, 5128, 2600), {"up": (256, "cut")}),
         ((133, 4608, 10608), {"up": (256, "tail")}),
         ((131, 5344, 4968), {"dh": (256, "cut")}),
         ((141, 4672, 19480), {"dh": (256, "tail")}),
         ((5, 2760, 22416), {"dh": (128, "tail")}),
         ((130, 4896, 5416), {"down": (256, "cut")}),
         ((269, 10168, 5056), {"down": (256, "tail")}),
         ((34, 624, 14144), {"down": (64, "cut"), "dh": (128, "whole")}),
         ((53, 8424, 672), {"down": (64, "whole")}),
         ((523, 64, 11936), {"dh": (256, "whole")}),
         ((705, 72, 5912), {"up": (256, "whole")}),
         ((394, 14728, 64), {"down": (256, "whole")})]


def test_the_sizes_take_every_way_of_the_gated_block():
    ways = {(launch, *way) for _, w in GATED for launch, way in w.items()}
    every = {(c, k) for c in (64, 128, 256) for k in ("whole", "cut", "tail")} - {(64, "tail")}
    assert {w for w in ways if w[0] == "up"} == {("up", *e) for e in every}
    assert {w for w in ways if w[0] == "dh"} == {("dh", *e) for e in every}
    assert {w for w in ways if w[0] == "down"} == {("down", *e) for e in every - {(128, "tail")}}


@pytest.mark.parametrize("size, ways", GATED)
def test_gated(size, ways):
    T, D, F = size
    for launch, way in ways.items():
        assert _way(gated_launch_shape(T, D, F, launch)) == way, launch
    i = gated._inputs(T, D, F, seed=3)
    if "up" in ways or "down" in ways:
        Y, G, U = gated._forward(i, "gelu_tanh")
        assert fg.sync_status() == 0
        gated._check_forward(i, "gelu_tanh", Y, G, U, True)
        del Y, G, U
    if "dh" in ways:
        got = gated._backward(i, "silu")
        assert fg.sync_status() == 0
        for g, w, t, name in zip(got, *gated._gradients(i, "silu"), ("dX", "dWg", "dWu", "dWd")):
            assert_close(g, w, (1 + U8) * t + U8 * w.abs(), name)


LOSS = [((1, 300, 4096), (64, "cut")), ((64, 1000, 4096), (64, "cut")), ((300, 1000, 1000), (64, "whole")),
        ((100, 5000, 4096), (128, "cut")), ((5, 21077, 2224), (128, "tail")), ((1, 9791, 64), (128, "whole")),
        ((130, 5259, 5840), (256, "cut")), ((133, 19881, 4984), (256, "tail")), ((1000, 20000, 1024), (256, "whole"))]


def test_the_sizes_take_every_way_of_the_loss():
    assert {w for _, w in LOSS} == {(c, k) for c in (64, 128, 256) for k in ("whole", "cut", "tail")} - {(64, "tail")}


@pytest.mark.parametrize("size, way", LOSS)
def test_loss(size, way):
    T, V, D = size
    for launch in ("stats", "g"):
        assert _way(loss_launch_shape(T, V, D, launch)) == way, launch
    x, w, t, dloss = loss._inputs(T, V, D, seed=2)
    out, lse = loss._forward(x, w, t)
    dX, dW = loss._backward(x, w, t, lse, dloss)
    assert fg.sync_status() == 0
    loss._check(x, w, t, dloss, out, lse, dX, dW)
    # and with the fused step at its end: dX from the weights as they were
    W, m, v, dX = w.clone(), *(torch.zeros(V, D, device="cuda") for _ in range(2)), torch.empty_like(x)
    fg.linear_cross_entropy_step(x, W, t, lse, dloss, dX, m, v, hp=Hparams(lr=1e-2, weight_decay=0.0), step=1)
    assert fg.sync_status() == 0
    loss._check(x, w, t, dloss, out, lse, dX, None)
    assert not torch.equal(W, w)
