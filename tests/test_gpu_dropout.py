"""Dropout on the GPU: the mask against the oracle's generator bit for bit, values against the formula."""
import math

import numpy as np
import pytest
import torch

import backward_optimizer_gb300 as fg
from oracle import philox
from tests.operators_reference import F64, U8, assert_close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _drops(n, p, seed, step, first=0):
    """Which of the elements first .. first+n-1 are dropped: the stated counter through the oracle's generator."""
    e = np.arange(first, first + n, dtype=np.uint64)
    j, m = e >> np.uint64(3), np.uint64(0xFFFFFFFF)
    ctr = np.stack([j & m, (j >> np.uint64(32)) + np.uint64(3 << 30), np.full(n, step & 0xFFFFFFFF, np.uint64),
                    np.full(n, step >> 32, np.uint64)])
    out = philox.philox4x32(ctr, (np.uint64(seed & 0xFFFFFFFF), np.uint64(seed >> 32)))
    word = out[((e >> np.uint64(1)) & np.uint64(3)).astype(np.intp), np.arange(n)]
    r16 = (word >> ((e & np.uint64(1)) * np.uint64(16)).astype(np.uint32)) & np.uint32(0xFFFF)
    return torch.from_numpy(r16 < round(p * 65536)).cuda()


def _want(x, res, p, seed, step):
    q = round(p * 65536)
    s = 65536 / (65536 - q) if q < 65536 else 0.0
    drop = _drops(x.numel(), p, seed, step).view(x.shape)
    y = torch.where(drop, 0.0, x.to(F64) * s)
    return (y if res is None else y + res.to(F64)), drop


def _check(y, want, x, dtype, p):
    # The scale s is rounded to binary32, off by at most 2^-24 s, and so is x s, by at most 2^-24 |x| s; then one fused
    # multiply-add, rounded once, to binary32, and for bf16 once more.  The result is off by (1 + h) 2^-24 |x| s +
    # h |want|, h the rounding's half step (bf16: both, below 2^-8 + 2^-23); |want| itself can be small beside the product.
    q = round(p * 65536)
    s = 65536 / (65536 - q) if q < 65536 else 0.0
    half = U8 + 2.0 ** -23 if dtype is torch.bfloat16 else 2.0 ** -24
    assert_close(y, want, half * want.abs() + (1 + half) * 2.0 ** -24 * s * x.to(F64).abs(), "y")


@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9,), (1, 4096), (3, 5, 17), (1023, 1001), (64, 8192), (8192 * 4 + 8,),
                                   (2, 8191)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.9999, 1.0])
@pytest.mark.parametrize("residual", [False, True])
def test_values_and_mask(shape, dtype, p, residual):
    gen = torch.Generator().manual_seed(math.prod(shape))
    x = torch.randn(shape, generator=gen).to(dtype).cuda()
    res = torch.randn(shape, generator=gen).to(dtype).cuda() if residual else None
    seed, step = 0x1234_5678_9ABC_DEF0, (1 << 40) + 3
    y = torch.full_like(x, 5.0)
    fg.dropout(x, y, p, seed=seed, step=step, residual=res)
    want, drop = _want(x, res, p, seed, step)
    _check(y, want, x, dtype, p)
    if not residual:
        assert torch.equal(y == 0, drop | (x == 0))
        dx = torch.empty_like(x)
        fg.dropout_backward(x, dx, p, seed=seed, step=step)
        assert torch.equal(dx, y)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [1, 4, 8])
def test_views_that_start_anywhere(dtype, shift):
    """Elements' own alignment is enough, and the mask does not depend on it."""
    n = 5003
    big = torch.randn(n + 16, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    x, out = big[shift:shift + n], torch.full((n + 16,), 3.0, dtype=dtype, device="cuda")
    y = out[shift:shift + n]
    fg.dropout(x, y, 0.3, seed=5, step=2, residual=x)
    aligned = torch.empty(n, dtype=dtype, device="cuda")
    fg.dropout(x.clone(), aligned, 0.3, seed=5, step=2, residual=x.clone())
    assert torch.equal(y, aligned)
    assert (out[:shift] == 3).all() and (out[shift + n:] == 3).all()


def test_in_place():
    x = torch.randn(3000, generator=torch.Generator().manual_seed(2)).cuda()
    r = torch.randn(3000, generator=torch.Generator().manual_seed(3)).cuda()
    want, over_x, over_r = torch.empty_like(x), x.clone(), r.clone()
    fg.dropout(x, want, 0.2, seed=1, residual=r)
    fg.dropout(over_x, over_x, 0.2, seed=1, residual=r)
    fg.dropout(x, over_r, 0.2, seed=1, residual=over_r)
    assert torch.equal(over_x, want) and torch.equal(over_r, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_dropped_element_may_be_anything(dtype):
    n = 10000
    drop = _drops(n, 0.4, 9, 1)
    x = torch.ones(n, dtype=dtype, device="cuda")
    x[drop] = torch.tensor([float("nan"), float("inf"), float("-inf")], device="cuda").to(dtype).repeat(n)[:int(drop.sum())]
    y = torch.empty_like(x)
    fg.dropout(x, y, 0.4, seed=9, step=1)
    assert torch.isfinite(y).all() and torch.equal(y == 0, drop)


def test_kept_share_and_independence():
    """Shares over 2^22 elements within six standard deviations; other seeds and steps, other masks."""
    n, p = 1 << 22, 0.25
    x = torch.ones(n, device="cuda")
    ys = []
    for seed, step in ((0, 0), (1, 0), (0, 1)):
        y = torch.empty_like(x)
        fg.dropout(x, y, p, seed=seed, step=step)
        ys.append(y == 0)
        assert abs(ys[-1].double().mean().item() - p) < 6 * (p * (1 - p) / n) ** 0.5
    for a, b in ((0, 1), (0, 2), (1, 2)):  # both dropped: p^2
        assert abs((ys[a] & ys[b]).double().mean().item() - p * p) < 6 * (p * p * (1 - p * p) / n) ** 0.5


def test_step_on_the_device_and_in_a_graph():
    x = torch.randn(4099, generator=torch.Generator().manual_seed(4)).cuda()
    step, y, want = torch.tensor([7], device="cuda"), torch.empty(4099, device="cuda"), torch.empty(4099, device="cuda")
    fg.dropout(x, y, 0.5, seed=3, step=step)
    fg.dropout(x, want, 0.5, seed=3, step=7)
    assert torch.equal(y, want)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fg.dropout(x, y, 0.5, seed=3, step=step)
        step += 1
    for k in (7, 8, 9):
        g.replay()
        fg.dropout(x, want, 0.5, seed=3, step=k)
        assert torch.equal(y, want), k


def test_elements_past_32_bits():
    """Element numbers over 2^32: a tensor of 4.3 billion elements, checked around the border and at its end."""
    n = (1 << 32) + 4096
    x = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    fg.dropout(x, x, 0.5, seed=11, step=5)
    for first in (0, (1 << 31) - 64, (1 << 32) - 64, n - 128):
        assert torch.equal(x[first:first + 128] == 0, _drops(128, 0.5, 11, 5, first))


def test_gradient_against_differences():
    """dropout is linear: dropout(x + d) - dropout(x) is what dropout_backward makes of d."""
    gen = torch.Generator().manual_seed(9)
    x, d = torch.randn(5000, generator=gen).cuda(), torch.randn(5000, generator=gen).cuda()
    y, y2, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    fg.dropout(x, y, 0.3, seed=4, step=2)
    fg.dropout(x + d, y2, 0.3, seed=4, step=2)
    fg.dropout_backward(d, dx, 0.3, seed=4, step=2)
    # x + d, two products by the scale (below 1.5) and their difference are rounded to binary32
    assert_close(dx, y2.to(F64) - y.to(F64), 8 * 2.0 ** -24 * (x.abs() + d.abs()).to(F64), "dx")
