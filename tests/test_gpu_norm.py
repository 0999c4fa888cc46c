"""Layer norm and RMS norm on the GPU against their formulas in binary64 (operators_reference.py)."""
import pytest
import torch

import backward_optimizer_gb300 as fg
from tests import operators_reference as ref
from tests.operators_reference import F64, U8, assert_close

pytestmark = pytest.mark.gpu

# A binary32 sum of n terms is off by at most n 2^-24 of the sum of magnitudes.  A thread adds up at most
# D / 512 runs of 8 terms (64 in registers), the group's join 32 + 5 more; 512 covers all sizes below.
S32 = 512 * 2.0 ** -24
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _inputs(T, D, dtype, w_dtype, seed, offset=0.5):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, D, generator=gen) * (0.5 + torch.rand(D, generator=gen)) + offset).to(dtype).cuda()
    w = (1 + 0.1 * torch.randn(D, generator=gen)).to(w_dtype).cuda()
    b = (0.1 * torch.randn(D, generator=gen)).to(w_dtype).cuda()
    dy = (0.01 * torch.randn(T, D, generator=gen)).to(dtype).cuda()
    add = (0.01 * torch.randn(T, D, generator=gen)).to(dtype).cuda()
    return x, w, b, dy, add


# one element, one token, rows of a warp, of several warps, of a block; vectors and scalars; rows that
# fit no registers (bf16 over 16384, fp32 over 8192, odd lengths over 4096)
SIZES = [(1, 1), (1, 4096), (3, 7), (5, 64), (33, 72), (257, 256), (64, 513), (16, 1001), (300, 2048), (9, 4100),
         (2, 8200), (7, 16384), (3, 20008), (4, 4099), (2, 70001), (1300, 136)]


def _check(T, D, dtype, kind, w_dtype=torch.float32, bias=True, eps=1e-5, seed=0, offset=0.5, with_add=False):
    dt = DTYPES[dtype]
    x, w, b, dy, add = _inputs(T, D, dt, w_dtype, seed, offset)
    layer = kind == "layer"
    bias = bias and layer
    y = torch.empty_like(x)
    mean = torch.empty(T, device="cuda") if layer else None
    rstd = torch.empty(T, device="cuda")
    fg.layer_norm(x, w, b if bias else None, y, mean, rstd, eps=eps, kind=kind)
    dx, dw = torch.empty_like(x), torch.empty(D, device="cuda")
    db = torch.empty(D, device="cuda") if layer else None
    fg.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, add if with_add else None, kind=kind)
    torch.cuda.synchronize()
    X, W, B, DY = x.to(F64), w.to(F64), b.to(F64), dy.to(F64)
    want, mu, r = ref.norm(X, W, B if bias else None, eps, kind)
    u = U8 if dtype == "bf16" else 0.0
    size = X.abs().mean(1, keepdim=True) if layer else torch.zeros_like(mu)
    # the mean's error, carried through x - mean; the variance's error is relative and of the same order,
    # but for the part of it that a wrong mean gives, the square of the mean's error
    d = S32 * (X.abs() + 2 * size)
    rel = S32 + (S32 * size * r) ** 2
    if layer:
        assert_close(mean[:, None], mu, S32 * size, "mean")
    assert_close(rstd[:, None], r, rel * r, "rstd")
    assert_close(y, want, (1 + u) * W.abs() * r * (d + rel * (X - mu).abs()) + S32 * want.abs() + u * want.abs(), "y")
    # the backward pass takes the library's own mean and rstd
    M, R = (mean[:, None].to(F64) if layer else mu), rstd[:, None].to(F64)
    gx, gw, gb = ref.norm_backward(DY, X, W, M, R, kind)
    xh = (X - M).abs() * R + S32 * (X.abs() + M.abs()) * R
    g = (DY * W).abs()
    tol = S32 * R * (g + g.mean(1, keepdim=True) + xh * (g * xh).mean(1, keepdim=True))
    if with_add:
        gx = gx + add.to(F64)
        tol = tol + S32 * add.to(F64).abs()
    assert_close(dx, gx, (1 + u) * tol + u * gx.abs(), "dx")
    n = (T + 512) * 2.0 ** -24  # the column's sum over tokens
    assert_close(dw, gw, n * (DY.abs() * xh).sum(0), "dweight")
    if layer:
        assert_close(db, gb, n * DY.abs().sum(0), "dbias")


@pytest.mark.parametrize("T, D", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_forward_and_backward(T, D, dtype, kind):
    _check(T, D, dtype, kind, eps=1e-5 if D > 1 else 1e-2)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("D", [512, 1001])
def test_bf16_weights_residual_gradient_no_bias(kind, D):
    _check(100, D, "bf16", kind, w_dtype=torch.bfloat16, bias=False, with_add=True)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_tokens_over_all_blocks(dtype):
    _check(5000, 320, dtype, "layer", seed=3)


def test_variance_is_taken_about_the_mean():
    """A mean 1000 times the deviation: E[x^2] - mean^2 would keep no digit of the variance in binary32."""
    T, D = 16, 1024
    gen = torch.Generator().manual_seed(1)
    x = (1000 + torch.randn(T, D, generator=gen)).cuda()
    w, y, rstd = torch.ones(D, device="cuda"), torch.empty(T, D, device="cuda"), torch.empty(T, device="cuda")
    fg.layer_norm(x, w, None, y, None, rstd)
    _, _, r = ref.norm(x.to(F64), w.to(F64), None, 1e-5, "layer")
    # the mean may be off by S32 * 1000 = 0.03 deviations, which enters the variance squared: 1e-3
    assert_close(rstd[:, None], r, 2e-3 * r, "rstd")


def test_constant_and_extreme_rows():
    D = 256
    rows = torch.zeros(6, D)
    rows[1] = 3.0          # variance 0
    rows[2, 0] = 1e30      # its square overflows binary32: y = 0 but for nothing finite to compare with
    rows[3, 5] = float("inf")
    rows[4, 7] = float("nan")
    rows[5, :] = torch.arange(D)
    x = rows.cuda()
    w, b = torch.ones(D, device="cuda"), torch.full((D,), 0.5, device="cuda")
    y = torch.empty_like(x)
    fg.layer_norm(x, w, b, y)
    torch.cuda.synchronize()
    assert torch.equal(y[0], b) and torch.equal(y[1], b)
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all()  # as the formula gives
    assert torch.isfinite(y[5]).all()  # rows do not touch one another


def test_gradient_against_differences():
    """(f(x + h) - f(x - h)) / 2h of f = sum(y c) in binary64 formulas fed by the library's forward."""
    T, D, h = 4, 96, 2.0 ** -6
    x, w, b, c, _ = _inputs(T, D, torch.float32, torch.float32, 5)
    for kind in ("layer", "rms"):
        bias = b if kind == "layer" else None
        mean = torch.empty(T, device="cuda") if kind == "layer" else None
        rstd, y = torch.empty(T, device="cuda"), torch.empty_like(x)
        fg.layer_norm(x, w, bias, y, mean, rstd, kind=kind)
        dx, dw = torch.empty_like(x), torch.empty(D, device="cuda")
        fg.layer_norm_backward(c, x, w, mean, rstd, dx, dw, torch.empty(D, device="cuda") if bias is not None else None,
                               kind=kind)

        def f(x, w):
            out = torch.empty_like(x)
            fg.layer_norm(x, w, bias, out, kind=kind)
            return (out.to(F64) * c.to(F64)).sum(1 if x.shape[0] == T else 0)

        for k in range(0, D, 17):
            e = torch.zeros(D, device="cuda")
            e[k] = h
            slope = (f(x + e, w) - f(x - e, w)) / (2 * h)
            # the difference's own error: h^2 f''' / 6 (f''' is below 20 |c| for these rows) and the
            # binary32 rounding of y, 2^-22 sum |y c| / 2h
            tol = 20 * h * h / 6 * c.abs().sum(1).to(F64) / D ** 0.5 + 2.0 ** -22 * (y * c).abs().sum(1).to(F64) / h
            assert_close(dx[:, k], slope, tol, f"dx, {kind}, column {k}")
            slope_w = ((f(x, w + e) - f(x, w - e)) / (2 * h)).sum()
            tol_w = 2.0 ** -22 * (y * c).abs().sum().to(F64) / h  # y is linear in w
            assert_close(dw[k], slope_w, tol_w, f"dweight, {kind}, column {k}")


def test_in_place_no_tokens_unaligned_and_streams():
    x, w, b, dy, add = _inputs(40, 512, torch.bfloat16, torch.float32, 9)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    fg.layer_norm(x, w, b, y, mean, rstd)
    dx, dw, db = torch.empty_like(x), torch.empty(512, device="cuda"), torch.empty(512, device="cuda")
    fg.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db)
    torch.cuda.synchronize()
    z = x.clone()
    fg.layer_norm(z, w, b, z)  # y may be x
    g = dy.clone()
    fg.layer_norm_backward(g, x, w, mean, rstd, g, dw.clone(), db.clone())  # dx may be dy
    torch.cuda.synchronize()
    assert torch.equal(z, y) and torch.equal(g, dx)
    # tensors that start one element past a 16-byte boundary take the scalar path: the same sums in
    # another order
    u = torch.empty(40 * 512 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(40, 512)
    u.copy_(x)
    v = torch.empty(40 * 512 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(40, 512)
    fg.layer_norm(u, w, b, v)
    torch.cuda.synchronize()
    assert_close(v, y.to(F64), 2 * U8 * y.to(F64).abs() + 1e-6, "y, unaligned")
    # another stream than the current one
    s = torch.cuda.Stream()
    y2, dw2, db2, dx2 = torch.empty_like(y), torch.empty_like(dw), torch.empty_like(db), torch.empty_like(dx)
    s.wait_stream(torch.cuda.current_stream())
    fg.layer_norm(x, w, b, y2, stream=s)
    fg.layer_norm_backward(dy, x, w, mean, rstd, dx2, dw2, db2, stream=s)
    s.synchronize()
    assert torch.equal(y2, y) and torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    # no tokens
    e = x[:0]
    dw.fill_(7)
    db.fill_(7)
    fg.layer_norm(e, w, b, e.clone())
    fg.layer_norm_backward(e, e, w, mean[:0], rstd[:0], e.clone(), dw, db)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


@pytest.mark.parametrize("T, D", [(33, 72), (5, 1001), (2, 70001)])
def test_nothing_outside_is_written(T, D):
    x, w, b, dy, _ = _inputs(T, D, torch.bfloat16, torch.float32, 2)
    buf = torch.full((T * D + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    red = torch.full((2 * D + 32,), 5.0, device="cuda")
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    y = buf[:T * D].view(T, D)
    fg.layer_norm(x, w, b, y, mean, rstd)
    fg.layer_norm_backward(dy, x, w, mean, rstd, y, red[:D], red[D:2 * D])
    torch.cuda.synchronize()
    assert (buf[T * D:] == 5).all() and (red[2 * D:] == 5).all()


def test_refusals():
    x, w, b, dy, _ = _inputs(8, 64, torch.bfloat16, torch.float32, 1)
    y, r = torch.empty_like(x), torch.empty(8, device="cuda")
    with pytest.raises(TypeError):
        fg.layer_norm(x.half(), w, b, y)
    with pytest.raises(TypeError):
        fg.layer_norm(x, w, b, y.float())
    with pytest.raises(TypeError):
        fg.layer_norm(x, w, b.bfloat16(), y)  # weight and bias share a type
    with pytest.raises(ValueError):
        fg.layer_norm(x, w[:32], b, y)
    with pytest.raises(ValueError):
        fg.layer_norm(x.t(), w[:8], b[:8], y.t())
    with pytest.raises(ValueError):
        fg.layer_norm(x, w, b, y, kind="batch")
    with pytest.raises(ValueError):
        fg.layer_norm(x.cpu(), w, b, y)
    with pytest.raises(ValueError):
        fg.layer_norm(x.view(2, 4, 64), w, b, y.view(2, 4, 64))
    for call in (lambda: fg.layer_norm(x, w, b, y, None, r, kind="rms"),   # an RMS norm has no bias
                 lambda: fg.layer_norm(x, w, None, y, r, r.clone(), kind="rms"),  # and no mean
                 lambda: fg.layer_norm(x, w, b, y, eps=-1.0),
                 lambda: fg.layer_norm_backward(dy, x, w, r, r, y, torch.empty(64, device="cuda"))):  # no dbias
        with pytest.raises(fg.ForgeError) as e:
            call()
        assert e.value.status == 1
    assert fg.sync_status() == 0
