"""Cases that time three more operators of a mixture-of-experts block:

- norm: root-mean-square norm with the residual's addition, its result in bf16 and in the e4m3 operand
  format of the grouped GEMMs, and its backward pass;
- balance: the router's balance loss and z loss of every sequence with its counts of every expert, and
  their gradient;
- lora: low-rank adapters of many requests, added to a projection's output.

`run` computes an operator in elementary torch operations, or, where `own` is true, by the
framework's calls.  `exact` is the same operator from its definition in 64 bits.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
E4M3, BF16, F32, I32, F64 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32, torch.float64
GROUP = 128
EPS = 1e-6

# ---------------------------------------------------------------- cases


def listed():
    return [
        # one decode step of one sequence, into the operand of an fp8 projection: latency alone
        dict(name="norm one token fp8", op="norm", T=1, K=7168, residual=True, y=False, fmt="km", weight="bfloat16"),
        # prompts in front of a layer: bf16 for the router and the dispatch, e4m3 for the shared expert
        dict(name="norm 4096 tokens", op="norm", T=4096, K=7168, residual=True, y=True, fmt="km", weight="bfloat16"),
        # a small model's rows of odd width and count, no residual
        dict(name="norm odd width", op="norm", T=8191, K=2047, residual=False, y=True, fmt=None, weight="float32"),
        # a training step's backward pass, the residual's gradient added
        dict(name="norm backward 4096 tokens", op="norm_backward", T=4096, K=7168, d_sum=True, weight="bfloat16"),
        # the same of a short ragged batch
        dict(name="norm backward 333 tokens", op="norm_backward", T=333, K=2048, d_sum=False, weight="float32"),
        # a training batch of 16 packed sequences over 256 experts, with the z loss
        dict(name="balance 256 experts 16 sequences", op="balance", T=8191, E=256, k=8, S=16, dtype="float32",
             score="softmax", z=True),
        # the router of the 64-expert workload: bf16 logits, one sum over the whole batch
        dict(name="balance 64 experts bf16", op="balance", T=4096, E=64, k=8, S=1, dtype="bfloat16", score="sigmoid",
             z=False),
        # every logit's gradient, on top of the one that the routing weights sent
        dict(name="balance backward 160 experts", op="balance_backward", T=8191, E=160, k=6, S=5, dtype="float32",
             score="softmax", z=True, add=True),
        # one decode step of one request
        dict(name="lora one token", op="lora", T=1, K=7168, N=4096, R=16, L=8, packed=False),
        # one decode step of 96 requests, each with an adapter of its own choice
        dict(name="lora 96 requests", op="lora", T=96, K=7168, N=4096, R=16, L=64, packed=False),
        # prompts of several requests in one batch
        dict(name="lora prompts", op="lora", T=4096, K=7168, N=4096, R=16, L=16, packed=True),
        # long ragged prompts, adapters of a higher rank
        dict(name="lora prompts rank 64", op="lora", T=8191, K=2048, N=7168, R=64, L=32, packed=True),
    ]


def _log_int(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def _log_mult(rng, lo, hi, m):
    return max(lo, _log_int(rng, lo, hi) // m * m)


def _draw_once(rng):
    op = rng.choice(["norm", "norm_backward", "balance", "balance_backward", "lora", "lora"])
    if op in ("norm", "norm_backward"):
        c = dict(op=op, T=_log_int(rng, 1, 8191), weight=rng.choice(["bfloat16", "float32"]))
        if op == "norm_backward":
            return dict(c, K=_log_int(rng, 64, 7168), d_sum=rng.random() < 0.7)
        fmt = rng.choice([None, "rows", "km", "km"])
        return dict(c, K=_log_int(rng, 64, 7168) if fmt is None else _log_mult(rng, 128, 7168, GROUP), fmt=fmt,
                    residual=rng.random() < 0.7, y=fmt is None or rng.random() < 0.5)
    if op in ("balance", "balance_backward"):
        E = _log_int(rng, 4, 512)
        c = dict(op=op, T=_log_int(rng, 1, 8191), E=E, k=rng.randint(1, min(16, E)), S=_log_int(rng, 1, 64),
                 dtype=rng.choice(["float32", "bfloat16"]), score=rng.choice(["softmax", "softmax", "sigmoid"]))
        c["z"] = c["score"] == "softmax" and rng.random() < 0.6
        return dict(c, add=rng.random() < 0.5) if op == "balance_backward" else c
    return dict(op=op, T=_log_int(rng, 1, 8191), K=_log_mult(rng, 256, 7168, 8), N=_log_mult(rng, 256, 7168, 8),
                R=rng.choice([8, 16, 16, 32, 64]), L=_log_int(rng, 1, 64), packed=rng.random() < 0.6)


def draw(rng):
    most = {k: max(work(c)[k] for c in listed()) for k in ("bytes", "flops")}
    while True:
        c = _draw_once(rng)
        if all(work(c)[k] <= most[k] for k in most):
            return c


# ---------------------------------------------------------------- inputs


def _gen(seed, k):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 64 + k)
    return g


def _randn(shape, seed, k, std=1.0):
    return torch.randn(shape, generator=_gen(seed, k), device=DEV) * std


def _empty(shape, dtype):
    """An output buffer with known contents where nothing is written."""
    return torch.zeros(shape, dtype=torch.uint8, device=DEV).view(dtype) if dtype is E4M3 \
        else torch.zeros(shape, dtype=dtype, device=DEV)


def _tokens(T, K, seed, k):
    """Hidden states: tokens of different size, a few columns much larger than the rest."""
    big = torch.exp(_randn((K,), seed, k, 0.5))
    row = torch.exp(_randn((T, 1), seed, k + 1, 0.5))
    return (_randn((T, K), seed, k + 2) * big * row).to(BF16)


def _weight(c, seed):
    return (1 + _randn((c["K"],), seed, 1, 0.1)).to(getattr(torch, c["weight"]))


def _offsets(c, seed):
    """Bounds of S sequences of very different lengths (some empty) over T tokens."""
    r = np.random.default_rng(int(seed))
    w = r.exponential(size=c["S"]) * (r.random(c["S"]) >= 0.1)
    w[int(r.integers(c["S"]))] += 1e-3
    n = r.multinomial(c["T"], w / w.sum())
    return torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=I32, device=DEV)


def _logits(c, seed):
    """Router logits: normal values on top of a fixed preference for some experts."""
    lean = _randn((c["E"],), seed, 1, 0.7)
    return (_randn((c["T"], c["E"]), seed, 2) + lean).to(getattr(torch, c["dtype"]))


def _adapters(c, seed):
    """The adapter of every row: popular ones often, a tenth of the rows without one; packed: requests of
    consecutive rows."""
    r = np.random.default_rng(int(seed))
    w = (1.0 + np.arange(c["L"])) ** -0.8
    w = r.permutation(w / w.sum())
    if c["packed"]:
        cuts = np.sort(r.integers(0, c["T"] + 1, size=min(c["T"], 2 * c["L"]) - 1))
        request = np.searchsorted(cuts, np.arange(c["T"]), side="right")
    else:
        request = np.arange(c["T"])
    of = r.choice(c["L"], size=int(request.max()) + 1, p=w)
    if len(of) > 1:
        of[r.random(len(of)) < 0.1] = -1
    return torch.tensor(of[request], dtype=I32, device=DEV)


def _scales(T, K, fmt):
    return _empty((T, K // GROUP) if fmt == "rows" else (K // GROUP, T), F32)


def prepare(case, seed):
    c, s = dict(case), {"case": dict(case)}
    op, T = c["op"], c["T"]
    if op == "norm":
        K = c["K"]
        s["x"], s["weight"] = _tokens(T, K, seed, 2), _weight(c, seed)
        s["residual"] = _tokens(T, K, seed, 5) if c["residual"] else None
        s["sum_out"] = _empty((T, K), BF16) if c["residual"] else None
        s["y"] = _empty((T, K), BF16) if c["y"] else None
        s["q"] = _empty((T, K), E4M3) if c["fmt"] else None
        s["q_scale"] = _scales(T, K, c["fmt"]) if c["fmt"] else None
        s["rstd"] = _empty((T,), F32)
        return s
    if op == "norm_backward":
        K = c["K"]
        s["h"], s["weight"] = _tokens(T, K, seed, 2), _weight(c, seed)
        s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + EPS).float()
        s["dy"] = _randn((T, K), seed, 5, 0.02).to(BF16)
        s["d_sum"] = _randn((T, K), seed, 6, 0.02).to(BF16) if c["d_sum"] else None
        s["dx"], s["d_weight"] = _empty((T, K), BF16), _empty((K,), F32)
        return s
    if op in ("balance", "balance_backward"):
        S, E = c["S"], c["E"]
        s["logits"] = _logits(c, seed)
        s["offsets"] = _offsets(c, seed) if S > 1 else None
        ids = torch.sort(s["logits"].float(), dim=1, descending=True, stable=True).indices[:, :c["k"]]
        if op == "balance":
            s["ids"] = ids.to(I32).contiguous()
            s["loss"], s["counts"], s["probs"] = _empty((S,), F32), _empty((S, E), I32), _empty((S, E), F32)
            s["z"] = _empty((S,), F32) if c["z"] else None
            return s
        at = (_sequence(s)[:, None] * E + ids).reshape(-1)
        s["counts"] = torch.bincount(at, minlength=S * E).reshape(S, E).to(I32)
        s["d_loss"] = 0.01 * torch.rand((S,), generator=_gen(seed, 4), device=DEV)
        s["d_z"] = 0.001 * torch.rand((S,), generator=_gen(seed, 5), device=DEV) if c["z"] else None
        s["before"] = _randn((T, E), seed, 6, 1e-5).to(s["logits"].dtype) if c["add"] else None
        s["d_logits"] = _empty((T, E), s["logits"].dtype)
        return s
    K, N, R, L = c["K"], c["N"], c["R"], c["L"]
    s["X"], s["Y"] = _randn((T, K), seed, 2).to(BF16), _randn((T, N), seed, 3).to(BF16)
    s["A"] = _randn((L, R, K), seed, 4, K ** -0.5).to(BF16)
    s["B"] = _randn((L, N, R), seed, 5, R ** -0.5).to(BF16)
    s["scale"] = 0.25 + torch.rand((L,), generator=_gen(seed, 6), device=DEV)
    s["adapter"] = _adapters(c, seed)
    s["used"] = sorted(set(s["adapter"].tolist()) - {-1})      # what a program's request table tells it
    s["out"] = _empty((T, N), BF16)
    return s


# ---------------------------------------------------------------- one pass


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# the framework's calls


def _mg():
    import moe_grouped_gemm_sizes_amd as mg
    return mg


def _workspace(s, make):
    """A workspace that a program keeps beside its buffers."""
    if "ws" not in s:
        s["ws"] = make()
    return s["ws"]


def _own_norm(s):
    _mg().rms_norm(s["x"], s["weight"], residual=s["residual"], sum_out=s["sum_out"], y=s["y"], q=s["q"],
                   q_scale=s["q_scale"], rstd=s["rstd"], eps=EPS, scale_km=s["case"]["fmt"] == "km")
    return {n: s[n] for n in ("sum_out", "y", "q", "q_scale", "rstd")}


def _own_norm_backward(s):
    mg, c = _mg(), s["case"]
    ws = _workspace(s, lambda: mg.rms_norm_workspace(c["T"], c["K"], s["dy"].device))
    mg.rms_norm_backward(s["dy"], s["h"], s["weight"], s["rstd"], s["dx"], s["d_weight"], ws, d_sum=s["d_sum"])
    return {"dx": s["dx"], "d_weight": s["d_weight"]}


def _score(mg, c):
    return mg.SCORE_SIGMOID if c["score"] == "sigmoid" else mg.SCORE_SOFTMAX


def _own_balance(s):
    mg, c = _mg(), s["case"]
    ws = _workspace(s, lambda: mg.balance_loss_workspace(c["T"], c["E"], c["S"], s["logits"].device))
    mg.balance_loss(s["logits"], s["ids"], s["loss"], s["counts"], ws, probs=s["probs"], z_loss=s["z"],
                    seq_offsets=s["offsets"], score=_score(mg, c))
    return {n: s[n] for n in ("loss", "z", "counts", "probs")}


def _own_balance_backward(s):
    mg, c = _mg(), s["case"]
    mg.balance_loss_backward(s["logits"], s["counts"], s["d_loss"], s["d_logits"], k=c["k"], d_z_loss=s["d_z"],
                             seq_offsets=s["offsets"], score=_score(mg, c), before=s["before"])
    return {"d_logits": s["d_logits"]}


def _own_lora(s):
    mg, c = _mg(), s["case"]
    ws = _workspace(s, lambda: mg.lora_workspace(c["T"], c["K"], c["R"], s["X"].device))
    mg.lora(s["X"], s["A"], s["B"], s["adapter"], s["Y"], s["out"], ws, scale=s["scale"])
    return {"out": s["out"]}


# the plain forms


def _quantize(v, fmt):
    """fp32 [T, K] -> e4m3 codes and fp32 scales of 1x128 groups."""
    g = v.reshape(v.shape[0], -1, GROUP)
    sc = g.abs().amax(-1) / 448.0
    sc = torch.where(sc > 0, sc, torch.ones_like(sc))
    q = (g / sc[..., None]).clamp(-448, 448).to(E4M3).reshape(v.shape)
    return q, sc if fmt == "rows" else sc.t().contiguous()


def _plain_norm(s):
    h = s["x"]
    if s["residual"] is not None:
        h = (h.float() + s["residual"].float()).to(BF16)
    f = h.float()
    rstd = 1 / torch.sqrt((f * f).mean(1) + EPS)
    v = f * rstd[:, None] * s["weight"].float()
    q, sc = _quantize(v, s["case"]["fmt"]) if s["case"]["fmt"] else (None, None)
    return {"sum_out": h if s["residual"] is not None else None, "y": v.to(BF16) if s["case"]["y"] else None, "q": q,
            "q_scale": sc, "rstd": rstd}


def _plain_norm_backward(s):
    dy, h, r = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    g = dy * s["weight"].float()
    xhat = h * r
    dx = r * (g - xhat * (g * xhat).mean(1, keepdim=True))
    if s["d_sum"] is not None:
        dx = dx + s["d_sum"].float()
    return {"dx": dx.to(BF16), "d_weight": (dy * xhat).sum(0, dtype=F64).float()}


def _sequence(s):
    """The sequence of every token."""
    T = s["case"]["T"]
    if s["offsets"] is None:
        return torch.zeros((T,), dtype=torch.long, device=DEV)
    t = torch.arange(T, device=DEV, dtype=I32)
    return (t[:, None] >= s["offsets"][None, 1:]).sum(1)


def _lengths(s):
    if s["offsets"] is None:
        return torch.full((1,), s["case"]["T"], device=DEV)
    return s["offsets"][1:] - s["offsets"][:-1]


def _probabilities(l, score):
    """(p, log-sum-exp, 1 - sigmoid) of logits."""
    m = l.amax(1, keepdim=True)
    if score == "softmax":
        e = torch.exp(l - m)
        z = e.sum(1, keepdim=True)
        return e / z, (m + torch.log(z))[:, 0], None
    sg = 1 / (1 + torch.exp(-l))
    return sg / sg.sum(1, keepdim=True), None, 1 / (1 + torch.exp(l))


def _plain_balance(s):
    c, seq = s["case"], _sequence(s)
    S, E, n = c["S"], c["E"], _lengths(s)
    p, lse, _ = _probabilities(s["logits"].float(), c["score"])
    # sums over a sequence's tokens as a product with its members (long sums: in 64 bits; counts are below 2^24)
    member = seq == torch.arange(S, device=DEV)[:, None]
    one = n.clamp(min=1).double()
    P = member.double() @ p.double() / one[:, None]
    has = torch.zeros_like(p).scatter_add_(1, s["ids"].long(), torch.ones(s["ids"].shape, device=DEV))
    counts = (member.float() @ has).to(I32)
    loss = (E / (c["k"] * one) * (counts * P).sum(1)).float()
    z = (member.double() @ (lse * lse).double() / one).float() if c["z"] else None
    return {"loss": loss, "z": z, "counts": counts, "probs": P.float()}


def _plain_balance_backward(s):
    c, seq = s["case"], _sequence(s)
    n = _lengths(s).clamp(min=1).float()
    p, lse, rest = _probabilities(s["logits"].float(), c["score"])
    g = ((c["E"] / c["k"]) * s["d_loss"] / (n * n))[:, None] * s["counts"].float()
    g = g[seq]
    d = p * (g - (p * g).sum(1, keepdim=True))
    if rest is not None:
        d = d * rest
    if s["d_z"] is not None:
        d = d + p * ((2 * s["d_z"] / n)[seq] * lse)[:, None]
    if s["before"] is not None:
        d = d + s["before"].float()
    return {"d_logits": d.to(s["logits"].dtype)}


def _plain_lora(s):
    out = s["Y"].clone()
    adapter = s["adapter"]
    for a in s["used"]:
        rows = torch.nonzero(adapter == a).reshape(-1)
        u = s["X"][rows].float() @ s["A"][a].float().t()
        out[rows] = (s["Y"][rows].float() + s["scale"][a] * (u @ s["B"][a].float().t())).to(BF16)
    return {"out": out}


# ---------------------------------------------------------------- work


def work(case):
    """Bytes of one pass, each input read once and each output written once; operations, roughly."""
    c, op, T = case, case["op"], case["T"]
    if op == "norm":
        K = c["K"]
        rows = 1 + 2 * c["residual"] + c["y"]
        q = T * K + 4 * T * (K // GROUP) if c["fmt"] else 0
        return {"bytes": 2 * T * K * rows + q + 4 * T + K * (2 if c["weight"] == "bfloat16" else 4), "flops": 8 * T * K}
    if op == "norm_backward":
        K = c["K"]
        return {"bytes": 2 * T * K * (3 + c["d_sum"]) + 4 * T + 4 * K + K * (2 if c["weight"] == "bfloat16" else 4),
                "flops": 12 * T * K}
    if op in ("balance", "balance_backward"):
        E, S = c["E"], c["S"]
        z = 4 if c["dtype"] == "float32" else 2
        if op == "balance":
            return {"bytes": T * E * z + 4 * T * c["k"] + 4 * S * (2 * E + 3), "flops": 10 * T * E}
        return {"bytes": T * E * z * (2 + c["add"]) + 4 * S * (E + 3), "flops": 15 * T * E}
    K, N, R = c["K"], c["N"], c["R"]
    used = min(c["L"], T)
    return {"bytes": 2 * T * K + 4 * T * N + 4 * T + used * 2 * R * (K + N), "flops": 2 * T * R * (K + N)}


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_norm(c, s):
    x = s["x"].double()
    h = x if s["residual"] is None else (x + s["residual"].double()).to(F32).to(BF16).double()
    rstd = (h.pow(2).sum(1) / c["K"] + EPS).pow(-0.5)
    v = s["weight"].double() * h * rstd[:, None]
    out = {"sum_out": h if s["residual"] is not None else None, "y": v if c["y"] else None, "q": None, "q_scale": None,
           "rstd": rstd}
    if c["fmt"]:
        a = v.reshape(c["T"], c["K"] // GROUP, GROUP).abs().max(2).values / 448
        a[a == 0] = 1
        out["q"] = (v.reshape(c["T"], -1, GROUP) / a[:, :, None]).reshape(c["T"], c["K"])
        out["q_scale"] = a if c["fmt"] == "rows" else a.t().contiguous()
    return out


def _exact_norm_backward(c, s):
    dy, h, w, r = s["dy"].double(), s["h"].double(), s["weight"].double(), s["rstd"].double()
    inner = torch.einsum("tk,tk->t", dy * w, h) / c["K"]
    dx = r[:, None] * dy * w - (r ** 3 * inner)[:, None] * h
    if s["d_sum"] is not None:
        dx += s["d_sum"].double()
    return {"dx": dx, "d_weight": (dy * h * r[:, None]).sum(0)}


def _bounds(c, s):
    if s["offsets"] is None:
        return [(0, c["T"])]
    o = s["offsets"].tolist()
    return list(zip(o[:-1], o[1:]))


def _exact_scores(l, score):
    if score == "softmax":
        return torch.softmax(l, 1), torch.logsumexp(l, 1)
    sg = torch.sigmoid(l)
    return sg / sg.sum(1, keepdim=True), None


def _exact_balance(c, s):
    S, E = c["S"], c["E"]
    l = s["logits"].double()
    loss, z = torch.zeros(S, dtype=F64, device=DEV), torch.zeros(S, dtype=F64, device=DEV)
    counts, probs = torch.zeros((S, E), dtype=I32, device=DEV), torch.zeros((S, E), dtype=F64, device=DEV)
    for i, (a, b) in enumerate(_bounds(c, s)):
        if b <= a:
            continue
        p, lse = _exact_scores(l[a:b], c["score"])
        counts[i] = torch.bincount(s["ids"][a:b].reshape(-1).long(), minlength=E).to(I32)
        f = counts[i].double() * E / (c["k"] * (b - a))
        probs[i] = p.mean(0)
        loss[i] = (f * probs[i]).sum()
        if c["z"]:
            z[i] = lse.square().mean()
    return {"loss": loss, "z": z if c["z"] else None, "counts": counts, "probs": probs}


def _exact_balance_backward(c, s):
    """By differentiating the definition."""
    l = s["logits"].double().clone().requires_grad_()
    total = torch.zeros((), dtype=F64, device=DEV)
    for i, (a, b) in enumerate(_bounds(c, s)):
        if b <= a:
            continue
        p, lse = _exact_scores(l[a:b], c["score"])
        f = s["counts"][i].double() * c["E"] / (c["k"] * (b - a))
        total = total + s["d_loss"][i].double() * (f * p.mean(0)).sum()
        if c["z"]:
            total = total + s["d_z"][i].double() * lse.square().mean()
    d, = torch.autograd.grad(total, l)
    return {"d_logits": d + s["before"].double() if s["before"] is not None else d}


def _exact_lora(c, s):
    out = s["Y"].double()
    for a in range(c["L"]):
        rows = torch.nonzero(s["adapter"] == a).reshape(-1)
        if len(rows):
            both = s["B"][a].double() @ (s["A"][a].double() @ s["X"][rows].double().t())
            out[rows] += float(s["scale"][a]) * both.t()
    return {"out": out}


def exact(case, seed):
    return globals()["_exact_" + case["op"]](case, prepare(case, seed))
