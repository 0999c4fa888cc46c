"""ForgeDropout's bookkeeping of masks, with a host function in place of the kernel (CPU only: no kernel is launched)."""
import copy
import pickle

import pytest
import torch
from torch.utils.checkpoint import checkpoint

from backward_optimizer_gb300 import blocks
from backward_optimizer_gb300.blocks import ForgeDropout

N = 4096


def _kept(n, p, seed, step):
    gen = torch.Generator("cpu").manual_seed(1000003 * seed + int(step))
    return torch.rand(n, generator=gen, dtype=torch.float32, device="cpu") >= p


@pytest.fixture(autouse=True)
def _on_the_host(monkeypatch):
    def dropout(x, y, p, seed=0, step=0, residual=None, stream=None):
        y.copy_(torch.where(_kept(x.numel(), p, seed, step).view(x.shape), x / (1 - p), 0.0))
        if residual is not None:
            y.add_(residual)

    monkeypatch.setattr(blocks.ops, "dropout", dropout)
    monkeypatch.setattr(blocks.ops, "dropout_backward",
                        lambda dy, dx, p, seed=0, step=0, stream=None: dropout(dy, dx, p, seed, step))


def _x(seed=0, n=N):
    return (torch.rand(n, generator=torch.Generator().manual_seed(seed)) + 0.5).requires_grad_()


def _mask_of(y):
    return y.detach() != 0


@pytest.mark.parametrize("reentrant", [True, False])
@pytest.mark.parametrize("behind", [False, True])
def test_a_recomputed_forward_takes_its_mask_again(reentrant, behind):
    """Two modules, one of them called twice, several forwards before the first backward, backwards in another order."""
    a, b = ForgeDropout(0.5, seed=1), ForgeDropout(0.25, seed=2)

    def region(x):
        y = b(a(a(x)))
        return y.square() if behind else y

    xs = [_x(i) for i in range(4)]
    ys = [checkpoint(region, x, use_reentrant=reentrant) for x in xs]
    assert (a.step, b.step) == (9, 5)
    masks = [_mask_of(y) for y in ys]
    assert not torch.equal(masks[0], masks[1])
    scale = 1 / (0.5 * 0.5 * 0.75)
    for i in (2, 0, 3, 1):
        ys[i].sum().backward()
        x = xs[i].detach()
        want = torch.where(masks[i], 2 * x * scale ** 2 if behind else torch.full_like(x, scale), 0.0)
        torch.testing.assert_close(xs[i].grad, want)
    assert (a.step, b.step) == (9, 5)  # recomputation takes no number
    y = b(a(a(xs[0])))
    assert (a.step, b.step) == (11, 6) and not torch.equal(_mask_of(y), masks[0])


@pytest.mark.parametrize("reentrant", [True, False])
def test_recomputed_twice_and_inside_another(reentrant):
    drop = ForgeDropout(0.5, seed=3)
    inner = lambda x: drop(x).square()  # noqa: E731
    x = _x()
    y = checkpoint(lambda t: checkpoint(inner, drop(t), use_reentrant=reentrant).sin(), x, use_reentrant=reentrant)
    kept = _mask_of(y)
    for _ in range(2 if not reentrant else 1):
        x.grad = None
        y.sum().backward(retain_graph=True)
        want = torch.where(kept, (4 * x.detach()).square().cos() * 32 * x.detach(), 0.0)
        torch.testing.assert_close(x.grad, want)
    assert drop.step == 3


def test_recomputed_without_its_generator_raises():
    drop = ForgeDropout(0.5, seed=3)
    x = _x()
    y = checkpoint(lambda t: drop(t).square(), x, use_reentrant=False, preserve_rng_state=False)
    with pytest.raises(RuntimeError, match="mask is not known"):
        y.sum().backward()


def test_two_forwards_from_one_state_of_the_generator():
    """Each takes a mask of its own; recomputing either could not tell which it is."""
    drop = ForgeDropout(0.5, seed=3)
    ys = []
    for i in range(2):
        torch.manual_seed(7)
        ys.append(checkpoint(lambda t: drop(t).square(), _x(), use_reentrant=False))
    assert not torch.equal(_mask_of(ys[0]), _mask_of(ys[1]))
    with pytest.raises(RuntimeError, match="mask is not known"):
        ys[1].sum().backward()
    # one that is through with its backward pass is not in the way: a generator seeded alike at each step
    drop = ForgeDropout(0.5, seed=4)
    for _ in range(3):
        torch.manual_seed(8)
        x = _x()
        y = checkpoint(lambda t: drop(t).square(), x, use_reentrant=False)
        kept = _mask_of(y)
        y.sum().backward()
        assert torch.equal(x.grad != 0, kept)
    assert drop.step == 4


def test_forwards_that_are_never_recomputed_are_forgotten():
    drop = ForgeDropout(0.5)
    x = _x(n=8)
    for _ in range(3000):
        drop(x)
    assert drop.step == 3001 and len(drop._masks) <= 1024
    y = checkpoint(lambda t: drop(t).square(), x, use_reentrant=False)
    kept = _mask_of(y)
    y.sum().backward()
    assert torch.equal(x.grad != 0, kept)


def test_default_device_and_type_do_not_matter():
    """The number that names a forward is the CPU generator's."""
    drop, x = ForgeDropout(0.5), _x()
    try:
        torch.set_default_device("meta")
        torch.set_default_dtype(torch.float64)
        y = drop(x)
    finally:
        torch.set_default_device(None)
        torch.set_default_dtype(torch.float32)
    assert torch.equal(_mask_of(y), _kept(N, 0.5, 0, 1))


@pytest.mark.parametrize("reentrant", [True, False])
@pytest.mark.parametrize("on_device", [False, True])
def test_the_step_that_the_caller_gives(reentrant, on_device):
    drop = ForgeDropout(0.5, seed=6)
    for k in (7, 7, 9):
        step, x = torch.tensor([k]) if on_device else k, _x()
        state = torch.get_rng_state()
        y = checkpoint(lambda t: drop(t, step=step).square(), x, use_reentrant=reentrant, preserve_rng_state=False)
        y.sum().backward()
        assert torch.equal(_mask_of(y), _kept(N, 0.5, 6, k)) and torch.equal(x.grad != 0, _mask_of(y))
        assert torch.equal(torch.get_rng_state(), state)  # such a forward draws no number
    assert drop.step == 1


def test_a_step_that_changes_before_the_backward_pass_raises():
    drop, step, x = ForgeDropout(0.5, seed=6), torch.tensor([3]), _x()
    y = drop(x, step=step)
    step += 1
    with pytest.raises(RuntimeError, match="step was changed"):
        y.sum().backward()
    with torch.inference_mode():
        assert torch.equal(_mask_of(drop(x, step=torch.tensor([4]))), _kept(N, 0.5, 6, 4))


@pytest.mark.parametrize("training", [True, False])
def test_what_is_refused_in_training_and_in_evaluation(training):
    drop, x = ForgeDropout(0.5).train(training), torch.ones(4, 8)
    for bad, residual in ((x.half(), None), (x.double(), None), (x.half(), x.half()), (x.long(), None), (x, x.bfloat16()),
                          (x.bfloat16(), x)):
        with pytest.raises(TypeError):
            drop(bad, residual=residual)
    for residual in (x[0], x[:, :1], torch.ones(()), x.view(8, 4), torch.ones(1, 4, 8), x.to("meta")):
        with pytest.raises(ValueError):
            drop(x, residual=residual)
    assert drop.step == 1 and not drop._masks  # a refused call takes no mask
    for t in (x, x.bfloat16()):
        assert drop(t, residual=t).dtype == t.dtype and drop(t).dtype == t.dtype
    if not training:
        assert drop(x) is x and torch.equal(drop(x, residual=x), x + x) and drop.step == 1


def test_modules_pickled_before_they_had_these_attributes():
    """A whole module that was pickled by an older version lacks what has been added since."""
    drop, head = ForgeDropout(0.5), blocks.ForgeHeadLoss(64, 64, device="cpu")
    for module, name in ((drop, "_masks"), (head, "reduction")):
        state = {k: v for k, v in module.__dict__.items() if k != name}
        old = type(module).__new__(type(module))
        old.__setstate__(state)
        assert getattr(old, name) == getattr(module, name)
    x = _x()
    old = ForgeDropout.__new__(ForgeDropout)
    old.__setstate__({k: v for k, v in drop.__dict__.items() if k != "_masks"})
    y = checkpoint(lambda t: old(t).square(), x, use_reentrant=False)
    y.sum().backward()
    assert torch.equal(x.grad != 0, _mask_of(y)) and not drop._masks


def test_copies_know_their_own_forwards():
    drop, x = ForgeDropout(0.5), _x()
    y = checkpoint(lambda t: drop(t).square(), x, use_reentrant=False)
    twin = pickle.loads(pickle.dumps(copy.deepcopy(drop)))
    for _ in range(2000):
        twin(x.detach())
    y.sum().backward()
    assert torch.equal(x.grad != 0, _mask_of(y)) and (drop.step, twin.step) == (2, 2002)


def test_what_draws_from_the_generator():
    drop, x = ForgeDropout(0.5), _x()
    state = torch.get_rng_state()
    drop(x).square().sum().backward()
    assert torch.equal(torch.get_rng_state(), state) and not drop._masks and drop.step == 2
    drop.eval()
    with torch.no_grad():
        drop(x)
    assert torch.equal(torch.get_rng_state(), state) and drop.step == 2
    drop.train()
    for reentrant in (True, False):
        with torch.random.fork_rng(devices=[]):
            checkpoint(drop, x, use_reentrant=reentrant)
            assert not torch.equal(torch.get_rng_state(), state)
    assert drop.step == 4 and len(drop._masks) == 1  # drawn from one state: which of the two it is cannot be told
    with pytest.raises(RuntimeError, match="mask is not known"):
        checkpoint(lambda t: drop(t).square(), x, use_reentrant=False, preserve_rng_state=False).sum().backward()


def test_plain_forwards_between_recomputed_ones():
    drop, xs = ForgeDropout(0.5), [_x(i) for i in range(3)]
    ys = []
    for x in xs:
        drop(x)
        ys.append(checkpoint(lambda t: drop(drop(t)).square(), x, use_reentrant=True))
        drop(x)
    for x, y in zip(xs, ys):
        kept = _mask_of(y)
        drop(x)
        y.sum().backward()
        assert torch.equal(x.grad != 0, kept)
    assert drop.step == 16
