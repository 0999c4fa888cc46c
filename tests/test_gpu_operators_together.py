"""The operators around the fused layers as a program runs them: captured in a CUDA graph, on several
streams at once, one after another without a wait between."""
import pytest
import torch

import backward_optimizer_gb300 as fg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    fg.build()
    fg.lib()


def _rand(gen, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=gen, device="cuda") * std).to(dtype)


class _Step:
    """norm -> gated block (+ residual) -> norm -> loss, and all gradients, into buffers of its own."""

    def __init__(self, T, D, F, V, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.x, self.w1, self.b1 = _rand(g, T, D), 1 + _rand(g, D, std=0.1, dtype=torch.float32), _rand(g, D, std=0.1, dtype=torch.float32)
        self.Wg, self.Wu, self.Wd = _rand(g, F, D, std=D ** -0.5), _rand(g, F, D, std=D ** -0.5), _rand(g, D, F, std=F ** -0.5)
        self.w2, self.W = 1 + _rand(g, D, std=0.1, dtype=torch.float32), _rand(g, V, D, std=D ** -0.5)
        self.t = torch.randint(V, (T,), generator=g, device="cuda")
        self.t[::7] = -100
        self.dloss = torch.full((T,), 1.0 / T, device="cuda")
        e = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
        f = torch.float32
        self.out = {"n1": e(T, D), "m1": e(T, dt=f), "r1": e(T, dt=f), "G": e(T, F), "U": e(T, F), "Y": e(T, D),
                    "n2": e(T, D), "r2": e(T, dt=f), "loss": e(T, dt=f), "lse": e(T, dt=f), "dn2": e(T, D), "dW": e(V, D),
                    "dY": e(T, D), "dw2": e(D, dt=f), "dn1": e(T, D), "dWg": e(F, D), "dWu": e(F, D), "dWd": e(D, F),
                    "dx": e(T, D), "dw1": e(D, dt=f), "db1": e(D, dt=f)}

    def run(self, stream=None):
        o = self.out
        fg.layer_norm(self.x, self.w1, self.b1, o["n1"], o["m1"], o["r1"], stream=stream)
        fg.gated_mlp(o["n1"], self.Wg, self.Wu, self.Wd, o["Y"], o["G"], o["U"], residual=self.x, stream=stream)
        fg.layer_norm(o["Y"], self.w2, None, o["n2"], None, o["r2"], kind="rms", stream=stream)
        fg.linear_cross_entropy(o["n2"], self.W, self.t, o["loss"], o["lse"], stream=stream)
        fg.linear_cross_entropy_backward(o["n2"], self.W, self.t, o["lse"], self.dloss, o["dn2"], o["dW"], stream=stream)
        fg.layer_norm_backward(o["dn2"], o["Y"], self.w2, None, o["r2"], o["dY"], o["dw2"], kind="rms", stream=stream)
        fg.gated_mlp_backward(o["dY"], o["n1"], o["G"], o["U"], self.Wg, self.Wu, self.Wd, o["dn1"], o["dWg"], o["dWu"], o["dWd"],
                              stream=stream)
        fg.layer_norm_backward(o["dn1"], self.x, self.w1, o["m1"], o["r1"], o["dx"], o["dw1"], o["db1"], add=o["dY"], stream=stream)

    def copy(self):
        return {k: v.clone() for k, v in self.out.items()}

    def clear(self):
        for v in self.out.values():
            v.fill_(float("nan"))


SHAPES = [(1, 256, 512, 1001), (3, 512, 1408, 5003), (300, 256, 704, 2049), (1100, 512, 1408, 3001)]


def _same(a, b):
    return [k for k in a if not torch.equal(a[k], b[k])]


@pytest.mark.parametrize("shape", SHAPES)
def test_a_captured_step_replays(shape):
    s = _Step(*shape, seed=1)
    s.run()
    torch.cuda.synchronize()
    want = s.copy()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        s.run()
    for _ in range(3):
        s.clear()
        graph.replay()
        torch.cuda.synchronize()
        assert fg.sync_status() == 0
        assert _same(s.out, want) == []


def test_without_waits_and_on_streams_at_once():
    steps = [_Step(*shape, seed=10 + i) for i, shape in enumerate(SHAPES)]
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.copy())
        s.clear()
    torch.cuda.synchronize()
    for _ in range(3):  # back to back on one stream: each launch may start before the last one ends
        for s in steps:
            s.run()
    torch.cuda.synchronize()
    assert fg.sync_status() == 0
    assert [_same(s.out, w) for s, w in zip(steps, want)] == [[]] * len(steps)
    for s in steps:
        s.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        for s, st in zip(steps, streams):
            s.run(stream=st)
    torch.cuda.synchronize()
    assert fg.sync_status() == 0
    assert [_same(s.out, w) for s, w in zip(steps, want)] == [[]] * len(steps)


def test_weights_written_just_before_they_are_read():
    """A block whose weights the stream's preceding work writes: a launch that starts early reads them as
    that work leaves them."""
    for T in (1, 2, 200):
        s = _Step(T, 1024, 2816, 300, seed=3)
        keep = [w.clone() for w in (s.Wg, s.Wu, s.Wd, s.W)]
        s.run()
        torch.cuda.synchronize()
        want = s.copy()
        for _ in range(5):
            for w, k in zip((s.Wg, s.Wu, s.Wd, s.W), keep):
                w.zero_()
            for w, k in zip((s.Wg, s.Wu, s.Wd, s.W), keep):
                w.copy_(k)
            s.run()
        torch.cuda.synchronize()
        assert _same(s.out, want) == []
