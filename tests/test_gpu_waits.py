"""Bounded waits of the ring kernels (norms, products of one to four tokens): one that runs out is reported,
the block arms no slot whose copies have not landed, and the calls behind it are right (needs a GB300)."""
import pytest
import torch

import backward_optimizer_gb300 as fg

pytestmark = pytest.mark.gpu

TIMEOUT = 6  # FORGE_ERR_TIMEOUT


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()
    assert fg.sync_status() == 0
    fg.set_wait_limit_ns(20_000_000)  # 20 ms
    yield
    fg.set_wait_limit_ns(2_000_000_000)
    fg.sync_status()


def _rand(seed, *shape, dtype=torch.bfloat16):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _check(call, outputs):
    """call() fills outputs: right, then with a stage withheld, then right again with the same bits."""
    call()
    assert fg.sync_status() == 0
    want = [t.clone() for t in outputs]
    fg.debug_withhold_next_stage()
    call()
    assert fg.sync_status() == TIMEOUT
    for t in outputs:
        t.fill_(0)
    call()
    assert fg.sync_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(outputs, want))


# rows that fill their rings many times over, several groups a block and one; a single row; a row for each slot
@pytest.mark.parametrize("T, D", [(5000, 512), (3000, 8192), (1, 4096), (400, 16384)])
@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norm(T, D, kind, dtype):
    if dtype is torch.float32:
        D //= 2  # the same bytes
    x, dy, add = (_rand(i, T, D, dtype=dtype) for i in range(3))
    w, b = _rand(4, D, dtype=torch.float32), _rand(5, D, dtype=torch.float32)
    layer = kind == "layer"
    y, rstd, mean = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda") if layer else None
    _check(lambda: fg.layer_norm(x, w, b if layer else None, y, mean, rstd, kind=kind), [y, rstd] + ([mean] if layer else []))
    dx, dw, db = torch.empty_like(x), torch.empty(D, device="cuda"), torch.empty(D, device="cuda") if layer else None
    _check(lambda: fg.layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, add, kind=kind),
           [dx, dw] + ([db] if layer else []))


# more groups of weight rows than slots, fewer than slots; a down projection whose ring fills before the wait
@pytest.mark.parametrize("T", [1, 2, 3, 4])
@pytest.mark.parametrize("D, F", [(1024, 8192), (64, 520), (4096, 4096)])
def test_few_token_products(T, D, F):
    X, R = _rand(0, T, D), _rand(1, T, D)
    Wg, Wu, Wd = (_rand(i, *s) * s[1] ** -0.5 for i, s in ((2, (F, D)), (3, (F, D)), (4, (D, F))))
    Y, G, U = torch.empty_like(X), *(torch.empty(T, F, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    _check(lambda: fg.gated_mlp(X, Wg, Wu, Wd, Y, G, U, residual=R), [Y, G, U])
