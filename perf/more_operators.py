"""Cases and plain forms of the operators that a model of experts, trained on preferences, needs next to the fused
layers.

Four operators, each forward and backward: products grouped by expert (a linear layer, and the gated feed-forward
block) over rows that lie sorted by expert in ragged runs; dropout on a residual branch, whose mask comes from a
counter and is never stored; and the preference loss of pairs of sequences, from the per-token losses that the
head's cross entropy leaves.  `run` is one pass: elementary torch operations in binary32 (sums over sequences in
binary64), rounded once at the end, or, with `own` true, the framework's kernels.  `exact` is the definition in
binary64.
"""
import math

import numpy as np
import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def listed():
    return [
        # one token of a served model through two of eight experts of the 4096/14336 block: the weights' bytes
        {"name": "experts fwd one token", "op": "gated_fwd", "R": 2, "E": 8, "active": 2, "tail": 0, "D": 4096, "F": 14336,
         "act": "silu", "save": False},
        # a small batch of a served model with many narrow experts: a few rows each, some with none
        {"name": "experts fwd 512 of 64", "op": "gated_fwd", "R": 512, "E": 64, "active": 60, "tail": 0, "D": 2048,
         "F": 1408, "act": "silu", "save": False},
        # a training batch through them, gate and up kept for the backward pass, some rows reserved and unused
        {"name": "experts fwd 32768 of 64", "op": "gated_fwd", "R": 32768, "E": 64, "active": 64, "tail": 1000, "D": 2048,
         "F": 1408, "act": "silu", "save": True},
        # the backward of the 4096/14336 block's experts: 4096 tokens, two experts each
        {"name": "experts bwd 8192 of 8", "op": "gated_bwd", "R": 8192, "E": 8, "active": 8, "tail": 0, "D": 4096,
         "F": 14336, "act": "silu"},
        # a ragged batch of a small model, three experts without a row
        {"name": "experts bwd 1003 of 16", "op": "gated_bwd", "R": 1003, "E": 16, "active": 13, "tail": 21, "D": 520,
         "F": 1032, "act": "gelu_tanh"},
        # a projection of its own for each of eight groups of tokens
        {"name": "expert linear fwd 4096 of 8", "op": "linear_fwd", "R": 4096, "E": 8, "active": 8, "tail": 0, "D": 4096,
         "F": 4096},
        # gradients of many narrow layers over a short batch
        {"name": "expert linear bwd 2048 of 32", "op": "linear_bwd", "R": 2048, "E": 32, "active": 31, "tail": 0,
         "D": 2048, "F": 1024},
        # the residual stream of a training batch at the widest model's width: bandwidth
        {"name": "dropout fwd 8192x5120", "op": "dropout_fwd", "T": 8192, "D": 5120, "p": 0.1, "dtype": "bf16"},
        # binary32 activations of a small model, a size that fits no vector
        {"name": "dropout bwd fp32 1023x1001", "op": "dropout_bwd", "T": 1023, "D": 1001, "p": 0.25, "dtype": "fp32"},
        # the smallest step of preference training: launches count
        {"name": "preference fwd 2 pairs", "op": "pref_fwd", "P": 2, "T": 515, "kind": "sigmoid", "mean": False,
         "mask": False},
        # a batch of pairs, prompts masked out
        {"name": "preference fwd 256 pairs", "op": "pref_fwd", "P": 256, "T": 262144, "kind": "sigmoid", "mean": False,
         "mask": True},
        # gradients of a few long sequences, averaged over their tokens
        {"name": "preference bwd 4 long pairs", "op": "pref_bwd", "P": 4, "T": 500001, "kind": "ipo", "mean": True,
         "mask": True},
    ]


def _log(rng, lo, hi, of=1):
    """A multiple of `of` between lo and hi, spread evenly over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / of)) * of))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(["gated_fwd", "gated_fwd", "gated_bwd", "gated_bwd", "linear_fwd", "linear_bwd", "dropout_fwd",
                         "dropout_bwd", "pref_fwd", "pref_bwd"])
        if op.startswith("gated") or op.startswith("linear"):
            R, E = _log(rng, 1, 32768), _log(rng, 1, 128)
            case = {"op": op, "R": R, "E": E, "active": min(R, rng.randint((E + 1) // 2, E)),
                    "tail": rng.choice([0, 0, rng.randint(1, 300)]), "D": _log(rng, 64, 5120, 8), "F": _log(rng, 64, 14336, 8)}
            if op.startswith("gated"):
                case["act"] = rng.choice(["silu", "gelu_tanh", "relu"])
            if op == "gated_fwd":
                case["save"] = rng.choice([True, False])
            if 3 * E * case["D"] * case["F"] > 8 * 3 * 4096 * 14336:  # weights of the listed cases at most
                continue
        elif op.startswith("dropout"):
            case = {"op": op, "T": _log(rng, 1, 8192), "D": _log(rng, 64, 5120, rng.choice([1, 8, 64])),
                    "p": rng.choice([0.05, 0.1, 0.25, 0.5]), "dtype": rng.choice(["bf16", "fp32"])}
        else:
            P = _log(rng, 1, 512)
            case = {"op": op, "P": P, "T": _log(rng, 4 * P, max(500001, 8 * P)),
                    "kind": rng.choice(["sigmoid", "hinge", "ipo"]), "mean": rng.choice([True, False]),
                    "mask": rng.choice([True, False])}
        if work(case)["flops"] <= most:
            return case


def work(case):
    op = case["op"]
    if op.startswith("gated") or op.startswith("linear"):
        R, E, A, D, F = case["R"], case["E"], case["active"], case["D"], case["F"]
        if op == "linear_fwd":  # X, the weights of experts with rows; Y
            return {"bytes": 2 * (R * (D + F) + A * D * F), "flops": 2 * R * D * F}
        if op == "linear_bwd":  # dY, X, those weights; dX, every dW
            return {"bytes": 2 * (R * (2 * D + F) + (A + E) * D * F), "flops": 4 * R * D * F}
        if op == "gated_fwd":  # X, three matrices of experts with rows; Y (G, U)
            return {"bytes": 2 * (2 * R * D + 3 * A * D * F + (2 * R * F if case["save"] else 0)), "flops": 6 * R * D * F}
        # dY, X, G, U, those matrices; dX, every dWg, dWu, dWd
        return {"bytes": 2 * (3 * R * D + 2 * R * F + 3 * (A + E) * D * F), "flops": 12 * R * D * F}
    if op.startswith("dropout"):
        n, size = case["T"] * case["D"], 2 if case["dtype"] == "bf16" else 4
        # x, residual; y, or dy; dx
        return {"bytes": n * size * (3 if op == "dropout_fwd" else 2), "flops": 2 * n}
    P, T = case["P"], case["T"]
    if op == "pref_fwd":  # nll, ref (mask), offsets; loss, reward, slope
        return {"bytes": T * (9 if case["mask"] else 8) + 4 * (2 * P + 1) + 4 * 5 * P, "flops": 2 * T}
    # (mask), offsets, slope, dloss; dnll
    return {"bytes": T * (5 if case["mask"] else 4) + 4 * (2 * P + 1) + 4 * 3 * P, "flops": T}


BETA, SMOOTHING, MARGIN = 0.1, 0.05, 0.0


def _ragged(total, parts, gen):
    """`parts` positive sizes of sum `total`, uneven: the lengths between sorted cuts, host numbers."""
    cuts = (torch.randperm(total - 1, generator=gen)[:parts - 1] + 1).sort().values.tolist()
    return [b - a for a, b in zip([0] + cuts, cuts + [total])]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)

    def normal(shape, std=1.0, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)

    op = case["op"]
    s = {"case": case}
    if op.startswith("gated") or op.startswith("linear"):
        R, E, A, D, F, rows = case["R"], case["E"], case["active"], case["D"], case["F"], case["R"] + case["tail"]
        # what a router leaves: some experts without a token, the others with shares of very different size
        sizes = [0] * E
        for e, n in zip(torch.randperm(E, generator=host)[:A].tolist(), _ragged(R, A, host)):
            sizes[e] = n
        s["sizes"] = sizes  # the plain form's; the framework's calls read the offsets on the device
        s["offsets"] = torch.tensor([0] + sizes).cumsum(0).to(torch.int32).cuda()
        s["X"] = normal((rows, D))
        if op.startswith("linear"):
            s["W"] = normal((E, F, D), 0.02)
            if op == "linear_fwd":
                s["Y"] = torch.zeros(rows, F, dtype=BF16, device="cuda")
            else:
                s["dY"] = normal((rows, F), 1e-3)
                s["dX"], s["dW"] = torch.zeros_like(s["X"]), torch.empty_like(s["W"])
            return s
        s["Wg"], s["Wu"], s["Wd"] = normal((E, F, D), 0.02), normal((E, F, D), 0.02), normal((E, D, F), 0.02)
        if op == "gated_fwd":
            s["Y"] = torch.zeros(rows, D, dtype=BF16, device="cuda")
            s["G"], s["U"] = ((torch.zeros(rows, F, dtype=BF16, device="cuda") for _ in range(2)) if case["save"]
                              else (None, None))
        else:
            s["dY"] = normal((rows, D), 1e-3)
            std = 0.02 * math.sqrt(D)  # what X Wg^T and X Wu^T of these inputs spread over
            s["G"], s["U"] = normal((rows, F), std), normal((rows, F), std)
            s["dX"] = torch.zeros_like(s["X"])
            s["dWg"], s["dWu"], s["dWd"] = (torch.empty_like(s[n]) for n in ("Wg", "Wu", "Wd"))
    elif op.startswith("dropout"):
        shape, dt = (case["T"], case["D"]), BF16 if case["dtype"] == "bf16" else F32
        s["seed"], s["step"] = seed * 0x9E3779B97F4A7C15 % 2**64, 1 + seed % 1000
        s["x" if op == "dropout_fwd" else "dy"] = normal(shape, 1.0, dt)
        s["residual"] = normal(shape, 1.0, dt) if op == "dropout_fwd" else None
        s["out"] = torch.empty(shape, dtype=dt, device="cuda")
    else:
        P, T = case["P"], case["T"]
        sizes = _ragged(T, 2 * P, host)
        offsets = torch.tensor([0] + sizes).cumsum(0)
        s["offsets"] = offsets.to(torch.int32).cuda()
        s["seq"] = torch.repeat_interleave(torch.arange(2 * P), torch.tensor(sizes)).cuda()  # the plain form's
        s["mask"] = None
        if case["mask"]:  # the prompt in front of each answer takes no part
            prompt = (torch.tensor(sizes).float() * 0.4 * torch.rand(2 * P, generator=host)).long()
            at = torch.arange(T) - torch.repeat_interleave(offsets[:-1], torch.tensor(sizes))
            s["mask"] = (at >= torch.repeat_interleave(prompt, torch.tensor(sizes))).cuda()
        if op == "pref_fwd":
            s["ref"] = torch.empty(T, device="cuda").exponential_(0.7, generator=gen)
            # a policy that has moved away from the reference, more on some sequences than on others
            s["nll"] = (s["ref"] + normal((T,), 0.1, F32) + normal((2 * P,), 0.01, F32)[s["seq"]]).clamp_min(0)
            s["loss"] = torch.empty(P, device="cuda")
            s["reward"], s["slope"] = torch.empty(2 * P, device="cuda"), torch.empty(2 * P, device="cuda")
        else:
            s["slope"] = normal((2 * P,), 0.05, F32)
            s["dloss"] = torch.full((P,), 1 / P, device="cuda")
            s["dnll"] = torch.empty(T, device="cuda")
    return s


# ------------------------------------------------------------------ one pass


def run(s):
    if own:
        return _run_own(s)
    return {"linear_fwd": _linear_fwd, "linear_bwd": _linear_bwd, "gated_fwd": _gated_fwd, "gated_bwd": _gated_bwd,
            "dropout_fwd": _dropout, "dropout_bwd": _dropout, "pref_fwd": _pref_fwd, "pref_bwd": _pref_bwd}[s["case"]["op"]](s)


def _run_own(s):
    import backward_optimizer_gb300 as fg
    c = s["case"]
    op = c["op"]
    if op == "linear_fwd":
        fg.expert_linear(s["X"], s["W"], s["offsets"], s["Y"])
        return {"Y": s["Y"]}
    if op == "linear_bwd":
        fg.expert_linear_backward(s["dY"], s["X"], s["W"], s["offsets"], s["dX"], s["dW"])
        return {"dX": s["dX"], "dW": s["dW"]}
    if op == "gated_fwd":
        fg.expert_gated_mlp(s["X"], s["Wg"], s["Wu"], s["Wd"], s["offsets"], s["Y"], s["G"], s["U"], act=c["act"])
        return {"Y": s["Y"], "G": s["G"], "U": s["U"]}
    if op == "gated_bwd":
        fg.expert_gated_mlp_backward(s["dY"], s["X"], s["G"], s["U"], s["Wg"], s["Wu"], s["Wd"], s["offsets"], s["dX"],
                                     s["dWg"], s["dWu"], s["dWd"], act=c["act"])
        return {"dX": s["dX"], "dWg": s["dWg"], "dWu": s["dWu"], "dWd": s["dWd"]}
    if op == "dropout_fwd":
        fg.dropout(s["x"], s["out"], c["p"], seed=s["seed"], step=s["step"], residual=s["residual"])
        return {"y": s["out"]}
    if op == "dropout_bwd":
        fg.dropout_backward(s["dy"], s["out"], c["p"], seed=s["seed"], step=s["step"])
        return {"dx": s["out"]}
    if op == "pref_fwd":
        fg.preference_loss(s["nll"], s["ref"], s["offsets"], s["loss"], s["reward"], s["slope"], mask=s["mask"], beta=BETA,
                           kind=c["kind"], smoothing=SMOOTHING if c["kind"] == "sigmoid" else 0.0, margin=MARGIN,
                           mean=c["mean"])
        return {"loss": s["loss"], "reward": s["reward"], "slope": s["slope"]}
    fg.preference_loss_backward(s["dloss"], s["slope"], s["offsets"], s["dnll"], mask=s["mask"])
    return {"dnll": s["dnll"]}


def _runs(s):
    """Each expert that has rows, and its rows."""
    at = 0
    for e, n in enumerate(s["sizes"]):
        if n:
            yield e, slice(at, at + n)
        at += n


def _linear_fwd(s):
    Y = torch.zeros_like(s["Y"])
    for e, r in _runs(s):
        Y[r] = (s["X"][r].float() @ s["W"][e].float().T).to(BF16)
    return {"Y": Y}


def _linear_bwd(s):
    dX, dW = torch.zeros_like(s["dX"]), torch.zeros_like(s["dW"])
    for e, r in _runs(s):
        dY = s["dY"][r].float()
        dX[r] = (dY @ s["W"][e].float()).to(BF16)
        dW[e] = (dY.T @ s["X"][r].float()).to(BF16)
    return {"dX": dX, "dW": dW}


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
    act, save = s["case"]["act"], s["case"]["save"]
    Y, G, U = (torch.zeros_like(s[n]) if s[n] is not None else None for n in ("Y", "G", "U"))
    for e, r in _runs(s):
        X = s["X"][r].float()
        g, u = X @ s["Wg"][e].float().T, X @ s["Wu"][e].float().T
        Y[r] = ((_act(g, act) * u) @ s["Wd"][e].float().T).to(BF16)
        if save:
            G[r], U[r] = g.to(BF16), u.to(BF16)
    return {"Y": Y, "G": G, "U": U}


def _gated_bwd(s):
    act = s["case"]["act"]
    dX, dWg, dWu, dWd = (torch.zeros_like(s[n]) for n in ("dX", "dWg", "dWu", "dWd"))
    for e, r in _runs(s):
        X, dY, G, U = (s[n][r].float() for n in ("X", "dY", "G", "U"))
        a = _act(G, act)
        dH = dY @ s["Wd"][e].float()
        dU, dG = dH * a, dH * U * _act_grad(G, act)
        dX[r] = (dG @ s["Wg"][e].float() + dU @ s["Wu"][e].float()).to(BF16)
        dWg[e], dWu[e], dWd[e] = (dG.T @ X).to(BF16), (dU.T @ X).to(BF16), (dY.T @ (a * U)).to(BF16)
    return {"dX": dX, "dWg": dWg, "dWu": dWu, "dWd": dWd}


# Philox4x32-10 (Salmon et al., SC'11): key = the seed's two words; counter = (e div 8 as 64 bits, the high word plus
# the stream's number times 2^30, step as 64 bits).  Element e takes the low (e even) or high (e odd) half of word
# (e div 2) mod 4, and is dropped where that number is below p 2^16.
_STREAM = 3  # 0 to 2 are the fused step's


def _drops(n, p, seed, step):
    m = 0xFFFFFFFF
    i = torch.arange((n + 7) // 8, device="cuda")
    c = [i & m, ((i >> 32) + (_STREAM << 30)) & m, torch.full_like(i, step & m), torch.full_like(i, step >> 32)]
    k = [seed & m, seed >> 32]
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((b >> 32) & m) ^ c[1] ^ k[0], b & m, ((a >> 32) & m) ^ c[3] ^ k[1], a & m]
        k = [(k[0] + 0x9E3779B9) & m, (k[1] + 0xBB67AE85) & m]
    halves = torch.stack([h for w in c for h in (w & 0xFFFF, w >> 16)], 1)
    return halves.reshape(-1)[:n] < round(p * 65536)


def _dropout(s):
    c = s["case"]
    x = (s["x"] if c["op"] == "dropout_fwd" else s["dy"]).float()
    kept = 65536 / (65536 - round(c["p"] * 65536))
    y = torch.where(_drops(x.numel(), c["p"], s["seed"], s["step"]).view(x.shape), 0, x * kept)
    if s["residual"] is not None:
        return {"y": (y + s["residual"].float()).to(s["out"].dtype)}
    return {"dx": y.to(s["out"].dtype)}


def _pref_fwd(s):
    c, P = s["case"], s["case"]["P"]
    d = s["ref"].double() - s["nll"].double()
    n = torch.ones_like(d)
    if s["mask"] is not None:
        d, n = torch.where(s["mask"], d, 0), s["mask"].double()
    total = torch.zeros(2 * P, dtype=F64, device="cuda").index_add_(0, s["seq"], d)
    count = torch.zeros(2 * P, dtype=F64, device="cuda").index_add_(0, s["seq"], n)
    per = 1 / count.clamp_min(1) if c["mean"] else torch.ones_like(count)
    score = total * per
    z = BETA * (score[:P] - score[P:]) - MARGIN
    if c["kind"] == "sigmoid":
        loss = (1 - SMOOTHING) * torch.log1p(torch.exp(-z.abs())) + (1 - SMOOTHING) * (-z).clamp_min(0) \
            + SMOOTHING * torch.log1p(torch.exp(-z.abs())) + SMOOTHING * z.clamp_min(0)
        g = 1 / (1 + torch.exp(-z)) - (1 - SMOOTHING)
    elif c["kind"] == "hinge":
        loss, g = (1 - z).clamp_min(0), torch.where(z < 1, -1.0, 0.0)
    else:
        loss, g = ((z - 0.5) / BETA) ** 2, 2 * (z - 0.5) / BETA**2
    slope = BETA * torch.cat([-g, g]) * per
    return {"loss": loss.float(), "reward": (BETA * score).float(), "slope": slope.float()}


def _pref_bwd(s):
    P = s["case"]["P"]
    g = (s["slope"] * torch.cat([s["dloss"], s["dloss"]]))[s["seq"]]
    return {"dnll": g if s["mask"] is None else torch.where(s["mask"], g, 0)}


# ------------------------------------------------------------------ the definitions in 64 bits


def _philox_halves(groups, seed, step):
    """The 16-bit numbers of `groups` counters, as an array [groups, 8]."""
    u, low, half = np.uint64, np.uint64(0xFFFFFFFF), np.uint64(32)
    index = np.arange(groups, dtype=u)
    x0, x1 = index & low, (index >> half) + u(_STREAM << 30)
    x2, x3 = np.full(groups, step & 0xFFFFFFFF, u), np.full(groups, step >> 32, u)
    for r in range(10):
        ka, kb = u((seed + r * 0x9E3779B9) & 0xFFFFFFFF), u(((seed >> 32) + r * 0xBB67AE85) & 0xFFFFFFFF)
        p, q = u(0xD2511F53) * x0, u(0xCD9E8D57) * x2
        x0, x1, x2, x3 = (q >> half) ^ x1 ^ ka, q & low, (p >> half) ^ x3 ^ kb, p & low
    return np.stack([x0, x1, x2, x3], 1).astype(np.uint32).view(np.uint16).reshape(groups, 8)


def exact(case, seed):
    if work(case)["flops"] > 1e13:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op.startswith("dropout"):
        x = s["x"] if op == "dropout_fwd" else s["dy"]
        n, at = x.numel(), int(np.rint(case["p"] * 65536))
        kept = torch.from_numpy(_philox_halves((n + 7) // 8, s["seed"], s["step"]).reshape(-1)[:n] >= at).cuda()
        y = torch.zeros(n, dtype=F64, device="cuda")
        y[kept] = x.reshape(-1)[kept].double() / (1 - at / 65536)
        y = y.view(x.shape)
        return {"y": y + s["residual"].double()} if op == "dropout_fwd" else {"dx": y}
    if op.startswith("pref"):
        P = case["P"]
        mask = s["mask"] if s["mask"] is not None else torch.ones(case["T"], dtype=torch.bool, device="cuda")
        cuts = s["offsets"].tolist()
        if op == "pref_bwd":
            dnll = torch.zeros(case["T"], dtype=F64, device="cuda")
            for i in range(2 * P):
                dnll[cuts[i]:cuts[i + 1]] = s["slope"][i].double() * s["dloss"][i % P].double()
            return {"dnll": dnll * mask}
        d = torch.cat([torch.zeros(1, dtype=F64, device="cuda"), torch.cumsum((s["ref"].double() - s["nll"].double()) * mask, 0)])
        k = torch.cat([torch.zeros(1, dtype=F64, device="cuda"), torch.cumsum(mask.double(), 0)])
        at = s["offsets"].long()
        total, count = d[at[1:]] - d[at[:-1]], (k[at[1:]] - k[at[:-1]]).clamp_min(1)
        score = (total / count if case["mean"] else total).requires_grad_()
        z = BETA * (score[:P] - score[P:]) - MARGIN
        if case["kind"] == "sigmoid":
            ls = torch.nn.functional.logsigmoid
            loss = -(1 - SMOOTHING) * ls(z) - SMOOTHING * ls(-z)
        elif case["kind"] == "hinge":
            loss = torch.relu(1 - z)
        else:
            loss = (z / BETA - 1 / (2 * BETA)) ** 2
        slope = -torch.autograd.grad(loss.sum(), score)[0]
        return {"loss": loss.detach(), "reward": BETA * score.detach(), "slope": slope / count if case["mean"] else slope}
    cuts = s["offsets"].tolist()
    v = {k: t.to(F64) if torch.is_tensor(t) and t.is_floating_point() and t.dim() == 2 else t for k, t in s.items()}
    zeros = {n: torch.zeros(s[n].shape, dtype=F64, device="cuda") for n in ("Y", "G", "U", "dX") if s.get(n) is not None}
    out = {"linear_fwd": ("Y",), "linear_bwd": ("dX", "dW"), "gated_fwd": ("Y", "G", "U"),
           "gated_bwd": ("dX", "dWg", "dWu", "dWd")}[op]
    o = {n: zeros[n] if n in zeros else torch.zeros(s[n].shape, dtype=F64, device="cuda") if s.get(n) is not None else None
         for n in out}
    for e in range(case["E"]):
        a, b = cuts[e], cuts[e + 1]
        if a == b:
            continue
        X = v["X"][a:b]
        if op.startswith("linear"):
            W = s["W"][e].double()
            if op == "linear_fwd":
                o["Y"][a:b] = torch.einsum("rd,fd->rf", X, W)
            else:
                o["dX"][a:b], o["dW"][e] = torch.einsum("rf,fd->rd", v["dY"][a:b], W), torch.einsum("rf,rd->fd", v["dY"][a:b], X)
            continue
        act = {"silu": torch.nn.functional.silu, "relu": torch.nn.functional.relu,
               "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[case["act"]]
        Wg, Wu, Wd = (s[n][e].double() for n in ("Wg", "Wu", "Wd"))
        if op == "gated_fwd":
            G, U = X @ Wg.T, X @ Wu.T
            o["Y"][a:b] = torch.einsum("rf,df->rd", act(G) * U, Wd)
            if case["save"]:
                o["G"][a:b], o["U"][a:b] = G, U
            continue
        G, U = v["G"][a:b].clone().requires_grad_(), v["U"][a:b].clone().requires_grad_()
        H = act(G) * U
        dG, dU = torch.autograd.grad(H, (G, U), v["dY"][a:b] @ Wd)
        o["dX"][a:b] = torch.cat([dG, dU], 1) @ torch.cat([Wg, Wu])
        o["dWg"][e], o["dWu"][e], o["dWd"][e] = dG.T @ X, dU.T @ X, v["dY"][a:b].T @ H.detach()
    return o
