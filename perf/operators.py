"""Cases and plain forms of the language-model operators around the fused layers.

Three operators, each with its backward pass: the norm (layer norm or RMS norm), the gated
feed-forward block, and the softmax cross entropy of a linear head over its vocabulary.  `run` is
one pass: elementary torch operations in binary32, rounded once at the end, or, with `own` true, the
framework's kernels.  `exact` is the definition in binary64.
"""
import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
EPS = 1e-5
IGNORE = -100  # the target of a token that takes no part in the loss


def listed():
    return [
        # one token on its way through a served model, width of the 4096-wide layers: latency
        {"name": "norm fwd one token", "op": "norm_fwd", "kind": "layer", "T": 1, "D": 4096, "dtype": "bf16"},
        # a training batch at the widest model's width: bandwidth
        {"name": "norm fwd rms 8192x5120", "op": "norm_fwd", "kind": "rms", "T": 8192, "D": 5120, "dtype": "bf16"},
        # the same in a layer's backward, weight and bias gradients included
        {"name": "norm bwd 4096x4096", "op": "norm_bwd", "kind": "layer", "T": 4096, "D": 4096, "dtype": "bf16"},
        # binary32 activations of a small model whose width fits no vector
        {"name": "norm bwd fp32 1023x1001", "op": "norm_bwd", "kind": "layer", "T": 1023, "D": 1001, "dtype": "fp32"},
        # one token through the feed-forward block of a served model: the weights' bytes
        {"name": "gated fwd one token", "op": "gated_fwd", "T": 1, "D": 4096, "F": 14336, "act": "silu", "save": False},
        # a training batch through the widest block, residual added, gate and up kept for the backward pass
        {"name": "gated fwd 8192 5120/17408", "op": "gated_fwd", "T": 8192, "D": 5120, "F": 17408, "act": "silu",
         "save": True},
        # the backward of the 4096/14336 block at its 4096 tokens
        {"name": "gated bwd 4096 4096/14336", "op": "gated_bwd", "T": 4096, "D": 4096, "F": 14336, "act": "silu"},
        # the smallest training step: launches count
        {"name": "gated bwd 256 256/512", "op": "gated_bwd", "T": 256, "D": 256, "F": 512, "act": "gelu_tanh"},
        # the loss of a training batch over a large vocabulary (evaluation reads no more than this)
        {"name": "loss fwd 4096 131072", "op": "loss_fwd", "T": 4096, "V": 131072, "D": 4096},
        # a ragged batch of a small model over an odd vocabulary
        {"name": "loss fwd 777 50001", "op": "loss_fwd", "T": 777, "V": 50001, "D": 1024},
        # gradients of that batch with respect to the hidden states and the head
        {"name": "loss bwd 4096 131072", "op": "loss_bwd", "T": 4096, "V": 131072, "D": 4096},
        # a short ragged batch over a small odd vocabulary
        {"name": "loss bwd 130 4099", "op": "loss_bwd", "T": 130, "V": 4099, "D": 512},
    ]


def _log(rng, lo, hi, of=1):
    """A multiple of `of` between lo and hi, spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / of)) * of))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["norm_fwd", "norm_bwd", "gated_fwd", "gated_bwd", "loss_fwd", "loss_bwd"])
        if op.startswith("norm"):
            case = {"op": op, "kind": rng.choice(["layer", "rms"]), "T": _log(rng, 1, 8192),
                    "D": _log(rng, 64, 8192, rng.choice([1, 8, 64])), "dtype": rng.choice(["bf16", "fp32"])}
        elif op.startswith("gated"):
            case = {"op": op, "T": _log(rng, 1, 8192), "D": _log(rng, 64, 5120, 8), "F": _log(rng, 64, 17408, 8),
                    "act": rng.choice(["silu", "gelu_tanh", "relu"])}
            if op == "gated_fwd":
                case["save"] = rng.choice([True, False])
        else:
            case = {"op": op, "T": _log(rng, 1, 8192), "V": _log(rng, 256, 160000), "D": _log(rng, 64, 5120, 8)}
        if work(case)["flops"] <= most:
            return case


def work(case):
    op, T, D = case["op"], case["T"], case["D"]
    if op.startswith("norm"):
        size, layer = (2 if case["dtype"] == "bf16" else 4), case["kind"] == "layer"
        if op == "norm_fwd":  # x; y; weight (bias); rstd (mean)
            return {"bytes": 2 * T * D * size + (1 + layer) * (4 * D + 4 * T), "flops": 8 * T * D}
        # dy, x; dx; weight; mean, rstd; dweight (dbias)
        return {"bytes": 3 * T * D * size + 4 * D + (1 + layer) * (4 * T + 4 * D), "flops": 14 * T * D}
    if op.startswith("gated"):
        F = case["F"]
        if op == "gated_fwd":  # X, R, Wg, Wu, Wd; Y (G, U)
            return {"bytes": 2 * (3 * T * D + 3 * D * F + (2 * T * F if case["save"] else 0)), "flops": 6 * T * D * F}
        # dY, X, G, U, Wg, Wu, Wd; dX, dWg, dWu, dWd
        return {"bytes": 2 * (3 * T * D + 2 * T * F + 6 * D * F), "flops": 12 * T * D * F}
    V = case["V"]
    if op == "loss_fwd":  # X, W, targets; loss, lse
        return {"bytes": 2 * (T * D + V * D) + 16 * T, "flops": 2 * T * V * D}
    # X, W, targets, lse, dloss; dX, dW
    return {"bytes": 4 * (T * D + V * D) + 16 * T, "flops": 6 * T * V * D}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std=1.0, dtype=BF16):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def empty(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    op, T, D = case["op"], case["T"], case["D"]
    s = {"case": case}
    if op.startswith("norm"):
        dt, layer = (BF16 if case["dtype"] == "bf16" else F32), case["kind"] == "layer"
        # a residual stream: channels of different size, and of a mean of their own
        s["x"] = (normal((T, D), 1.0, F32) * (0.5 + torch.rand(D, generator=gen, device="cuda"))
                  + 0.3 * normal((D,), 1.0, F32)).to(dt)
        s["w"] = 1.0 + normal((D,), 0.1, F32)
        s["b"] = normal((D,), 0.1, F32) if layer else None
        if op == "norm_fwd":
            s["y"], s["rstd"] = empty(T, D, dtype=dt), empty(T, dtype=F32)
            s["mean"] = empty(T, dtype=F32) if layer else None
        else:
            s["dy"] = normal((T, D), 1e-2, dt)
            x = s["x"].float()  # what the forward pass left
            s["mean"] = x.mean(1) if layer else None
            s["rstd"] = 1 / ((x - s["mean"][:, None] if layer else x).square().mean(1) + EPS).sqrt()
            s["dx"], s["dw"] = empty(T, D, dtype=dt), empty(D, dtype=F32)
            s["db"] = empty(D, dtype=F32) if layer else None
    elif op.startswith("gated"):
        F = case["F"]
        s["X"] = normal((T, D))
        s["Wg"], s["Wu"] = normal((F, D), 0.02), normal((F, D), 0.02)
        s["Wd"] = normal((D, F), 0.02)
        if op == "gated_fwd":
            s["R"], s["Y"] = normal((T, D)), empty(T, D)
            s["G"], s["U"] = (empty(T, F), empty(T, F)) if case["save"] else (None, None)
        else:
            s["dY"] = normal((T, D), 1e-3)
            std = 0.02 * math.sqrt(D)  # what X Wg^T and X Wu^T of these inputs spread over
            s["G"], s["U"] = normal((T, F), std), normal((T, F), std)
            s["dX"], s["dWg"], s["dWu"], s["dWd"] = empty(T, D), empty(F, D), empty(F, D), empty(D, F)
    else:
        V = case["V"]
        s["X"], s["W"] = normal((T, D)), normal((V, D), 0.02)
        target = torch.randint(V, (T,), generator=gen, device="cuda")
        out = torch.rand(T, generator=gen, device="cuda") < 0.05  # padding and prompts: no loss
        s["target"] = torch.where(out, IGNORE, target)
        if op == "loss_fwd":
            s["loss"], s["lse"] = empty(T, dtype=F32), empty(T, dtype=F32)
        else:
            # what the forward pass left, and the mean over the tokens that count
            s["lse"] = torch.cat([torch.logsumexp((x @ s["W"].T).float(), 1) for x in s["X"].split(1024)])
            s["dloss"] = (~out).float() / max(1, int((~out).sum()))
            s["dX"], s["dW"] = empty(T, D), empty(V, D)
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _run_own(s)
    return {"norm_fwd": _norm_fwd, "norm_bwd": _norm_bwd, "gated_fwd": _gated_fwd, "gated_bwd": _gated_bwd,
            "loss_fwd": _loss_fwd, "loss_bwd": _loss_bwd}[s["case"]["op"]](s)


def _run_own(s):
    import backward_optimizer_gb300 as fg
    op = s["case"]["op"]
    if op == "norm_fwd":
        fg.layer_norm(s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"], eps=EPS, kind=s["case"]["kind"])
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "norm_bwd":
        fg.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"],
                               kind=s["case"]["kind"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "gated_fwd":
        fg.gated_mlp(s["X"], s["Wg"], s["Wu"], s["Wd"], s["Y"], s["G"], s["U"], residual=s["R"], act=s["case"]["act"])
        return {"Y": s["Y"], "G": s["G"], "U": s["U"]}
    if op == "gated_bwd":
        fg.gated_mlp_backward(s["dY"], s["X"], s["G"], s["U"], s["Wg"], s["Wu"], s["Wd"], s["dX"], s["dWg"], s["dWu"],
                              s["dWd"], act=s["case"]["act"])
        return {"dX": s["dX"], "dWg": s["dWg"], "dWu": s["dWu"], "dWd": s["dWd"]}
    if op == "loss_fwd":
        fg.linear_cross_entropy(s["X"], s["W"], s["target"], s["loss"], s["lse"], ignore_index=IGNORE)
        return {"loss": s["loss"], "lse": s["lse"]}
    fg.linear_cross_entropy_backward(s["X"], s["W"], s["target"], s["lse"], s["dloss"], s["dX"], s["dW"],
                                     ignore_index=IGNORE)
    return {"dX": s["dX"], "dW": s["dW"]}


def _norm_fwd(s):
    x = s["x"].float()
    mean = x.mean(1) if s["b"] is not None else None
    c = x - mean[:, None] if mean is not None else x
    rstd = torch.rsqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * s["w"]
    if s["b"] is not None:
        y = y + s["b"]
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    c = x - s["mean"][:, None] if s["mean"] is not None else x
    xh = c * s["rstd"][:, None]
    g = dy * s["w"]
    dx = g - xh * (g * xh).mean(1, keepdim=True)
    if s["mean"] is not None:
        dx = dx - g.mean(1, keepdim=True)
    dx = dx * s["rstd"][:, None]
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0), "db": dy.sum(0) if s["mean"] is not None else None}


_C = math.sqrt(2 / math.pi)


def _act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    if act == "relu":
        return torch.where(g > 0, g, 0)
    return 0.5 * g * (1 + torch.tanh(_C * (g + 0.044715 * g * g * g)))


def _act_grad(g, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-g))
        return p * (1 + g * (1 - p))
    if act == "relu":
        return (g > 0).to(g.dtype)
    t = torch.tanh(_C * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * _C * (1 + 3 * 0.044715 * g * g)


def _gated_fwd(s):
    X = s["X"].float()
    G, U = X @ s["Wg"].float().T, X @ s["Wu"].float().T
    Y = (_act(G, s["case"]["act"]) * U) @ s["Wd"].float().T + s["R"].float()
    save = s["case"]["save"]
    return {"Y": Y.to(BF16), "G": G.to(BF16) if save else None, "U": U.to(BF16) if save else None}


def _gated_bwd(s):
    act = s["case"]["act"]
    X, dY, G, U = s["X"].float(), s["dY"].float(), s["G"].float(), s["U"].float()
    a = _act(G, act)
    dH = dY @ s["Wd"].float()
    dU, dG = dH * a, dH * U * _act_grad(G, act)
    dX = dG @ s["Wg"].float() + dU @ s["Wu"].float()
    return {"dX": dX.to(BF16), "dWg": (dG.T @ X).to(BF16), "dWu": (dU.T @ X).to(BF16),
            "dWd": (dY.T @ (a * U)).to(BF16)}


def _loss_fwd(s):
    logits = s["X"].float() @ s["W"].float().T
    top = logits.max(1, keepdim=True).values
    lse = (logits - top).exp().sum(1).log() + top[:, 0]
    counts = s["target"] != IGNORE
    at = logits.gather(1, torch.where(counts, s["target"], 0)[:, None])[:, 0]
    return {"loss": torch.where(counts, lse - at, 0), "lse": lse}


def _loss_bwd(s):
    X, W = s["X"].float(), s["W"].float()
    counts = s["target"] != IGNORE
    g = (X @ W.T - s["lse"][:, None]).exp()
    rows = torch.arange(g.shape[0], device=g.device)
    g[rows, torch.where(counts, s["target"], 0)] -= 1
    g = g * torch.where(counts, s["dloss"], 0)[:, None]
    return {"dX": (g @ W).to(BF16), "dW": (g.T @ X).to(BF16)}


# ------------------------------------------------------------------ the definitions in 64 bits


def exact(case, seed):
    if work(case)["flops"] > 2e13:
        return None
    s = prepare(case, seed)
    op = case["op"]
    v = {k: t.to(F64) if torch.is_tensor(t) and t.is_floating_point() else t for k, t in s.items()}
    if op == "norm_fwd":
        x, layer = v["x"], case["kind"] == "layer"
        mean = x.sum(1) / case["D"] if layer else torch.zeros_like(x[:, 0])
        rstd = (((x - mean[:, None]) ** 2).sum(1) / case["D"] + EPS) ** -0.5
        y = torch.einsum("td,t,d->td", x - mean[:, None], rstd, v["w"])
        return {"y": y + v["b"] if layer else y, "mean": mean if layer else None, "rstd": rstd}
    if op == "norm_bwd":
        layer, D = case["kind"] == "layer", case["D"]
        xh = (v["x"] - (v["mean"][:, None] if layer else 0)) * v["rstd"][:, None]
        g = v["dy"] * v["w"]
        # the Jacobian of xh takes out of g its part along xh, and for the layer norm its mean
        along = torch.einsum("td,td->t", g, xh) / D
        flat = g.sum(1) / D if layer else torch.zeros_like(along)
        dx = (g - flat[:, None] - along[:, None] * xh) * v["rstd"][:, None]
        return {"dx": dx, "dw": torch.einsum("td,td->d", v["dy"], xh), "db": v["dy"].sum(0) if layer else None}
    if op.startswith("gated"):
        act = {"silu": torch.nn.functional.silu, "relu": torch.nn.functional.relu,
               "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[case["act"]]
        if op == "gated_fwd":
            G, U = v["X"] @ v["Wg"].T, v["X"] @ v["Wu"].T
            save = case["save"]
            return {"Y": torch.addmm(v["R"], act(G) * U, v["Wd"].T), "G": G if save else None,
                    "U": U if save else None}
        G, U = v["G"].requires_grad_(), v["U"].requires_grad_()
        H = act(G) * U
        dG, dU = torch.autograd.grad(H, (G, U), v["dY"] @ v["Wd"])
        return {"dX": torch.cat([dG, dU], 1) @ torch.cat([v["Wg"], v["Wu"]]), "dWg": dG.T @ v["X"],
                "dWu": dU.T @ v["X"], "dWd": v["dY"].T @ H.detach()}
    keep = s["target"] >= 0
    if op == "loss_fwd":
        loss, lse = [], []
        for x, t in zip(v["X"].split(512), s["target"].split(512)):
            logp = torch.nn.functional.log_softmax(l := x @ v["W"].T, 1)
            loss.append(torch.nn.functional.nll_loss(logp, t, ignore_index=IGNORE, reduction="none"))
            lse.append(torch.logsumexp(l, 1))
        return {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    dX, dW = torch.empty_like(v["X"]), torch.zeros_like(v["W"])
    for i in range(0, case["T"], 512):
        x, k = v["X"][i:i + 512], keep[i:i + 512]
        p = torch.exp(x @ v["W"].T - v["lse"][i:i + 512, None])
        hot = torch.zeros_like(p)
        hot[k.nonzero()[:, 0], s["target"][i:i + 512][k]] = 1
        g = (p - hot) * (v["dloss"][i:i + 512] * k)[:, None]
        dX[i:i + 512] = g @ v["W"]
        dW += g.T @ x
    return {"dX": dX, "dW": dW}
