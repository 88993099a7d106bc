"""The router's balance loss and its gradient on MI355X against the fp64 oracle (oracle/block.py).

Bounds, with u = 2^-24 (half a step of fp32) and D the distance of a logit from its token's largest:
- p: e^x of a rounded difference x is off by |x| u + 2 u, a sum of E terms in tree order by less than 16 u, the
  reciprocal and the product by u each; sigmoids add a division and a second exponential: rel <= (D + 26) 2 u.
- P: tokens of a tile in a lane's chain, 6 steps, 4 waves (terms of one sign): (tile + 12) u more, then 64 bits.
- ln sum e^l: the sum's relative error (20 + D of its large terms, which is small: 64 u in all) and 2 u of the value.
- d_logits: g = d_loss E c / (k n^2) is off by 6 u, <p, g> by p's error and 16 u of the terms; 1 - sigmoid by
  (|l| + 4) 2 u; bf16 rounds by 2^-8 of the result.
Values below 2^-126 may be lost.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from oracle import block as ob
from tests.test_gpu_layer import SENTINEL, U, buf, f64, gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
TINY = 2.0 ** -126


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def code(score):
    return mg.SCORE_SIGMOID if score == "sigmoid" else mg.SCORE_SOFTMAX


def tile(T):
    t = (T + 255) // 256
    return 32 if t <= 32 else (t + 15) // 16 * 16


def distance(l):
    c = ob.clean(l)
    m = c.max(axis=1, keepdims=True)
    d = np.where(c > -np.inf, np.where(m > -np.inf, m, 0) - np.where(c > -np.inf, c, 0), 0)
    return np.minimum(d, 200.0)                              # e^-200 is 0 on both sides of TINY


def p_error(l):
    """Relative error of every p, and the absolute one of the log-sum-exp."""
    return (distance(l) + 26) * 2 * U, 64 * U + 2 * U * np.abs(ob.log_sum_exp(l))


def inputs(T, E, k, S, kind, seed, std=1.0):
    g = gen(seed)
    l = (torch.randn(T, E, generator=g) * std + torch.randn(E, generator=g)).to(kind)
    ids = torch.randint(-1, E + 1, (T, k), generator=g).to(I32)      # some are none
    if S == 0:
        return l, ids, None
    cut = torch.sort(torch.randint(0, T + 1, (S + 1,), generator=g)).values
    return l, ids, cut.to(I32)


def forward(l, ids, off, score, z=True, probs=True, ws=None, stream=None):
    T, E = l.shape
    S = 1 if off is None else len(off) - 1
    out = dict(loss=buf((S,), F32), z=buf((S,), F32) if z else None, counts=buf((S, E), I32),
               probs=buf((S, E), F32) if probs else None)
    dev = [None if v is None else v.cuda() for v in (l, ids, off)]
    mg.balance_loss(dev[0], dev[1], out["loss"], out["counts"], mg.balance_loss_workspace(T, E, S) if ws is None else ws,
                    probs=out["probs"], z_loss=out["z"], seq_offsets=dev[2], score=code(score), stream=stream)
    torch.cuda.synchronize()
    return out


def check_forward(l, ids, off, score, **kw):
    z = score == "softmax"
    got = forward(l, ids, off, score, z=z, **kw)
    L, (T, E), k = l.double().numpy(), l.shape, ids.shape[1]
    loss, zz, counts, probs = ob.balance_loss(L, ids.numpy(), None if off is None else off.tolist(), score)
    assert np.array_equal(got["counts"].cpu().numpy(), counts)
    ep, else_ = p_error(L)
    p, lse = ob.probabilities(L, score), ob.log_sum_exp(L)
    for s, (a, b) in enumerate(ob.bounds(None if off is None else off.tolist(), T)):
        n = max(b - a, 1)
        chain = (min(tile(T), n) + 12) * U
        err = (p[a:b] * ep[a:b] + TINY).sum(0) / n + (chain + U) * probs[s] if b > a else np.zeros(E)
        if got["probs"] is not None:
            assert (np.abs(f64(got["probs"])[s] - probs[s]) <= err).all(), s
        lim = E / (k * n) * (counts[s] * err).sum() + U * loss[s]
        assert abs(float(got["loss"][s]) - loss[s]) <= lim, (s, float(got["loss"][s]), loss[s], lim)
        if z and zz[s] > torch.finfo(F32).max:               # past fp32's range
            assert float(got["z"][s]) == float("inf")
        elif z:
            e = (2 * np.abs(lse[a:b]) * else_[a:b] + else_[a:b] ** 2).sum() / n + (chain + 3 * U) * zz[s]
            assert abs(float(got["z"][s]) - zz[s]) <= e, (s, float(got["z"][s]), zz[s], e)
    return got


def check_backward(l, ids, off, score, seed, add=True, z=True):
    T, E = l.shape
    k, S = ids.shape[1], 1 if off is None else len(off) - 1
    g = gen(seed + 100)
    offs = None if off is None else off.tolist()
    counts = ob.balance_loss(l.double().numpy(), ids.numpy(), offs, score)[2]
    dl, dz = torch.randn(S, generator=g), torch.randn(S, generator=g) if z and score == "softmax" else None
    before = torch.randn(T, E, generator=g).to(l.dtype) if add else None
    d = buf((T, E), l.dtype)
    mg.balance_loss_backward(l.cuda(), torch.from_numpy(counts).to(I32).cuda(), dl.cuda(), d, k=k,
                             d_z_loss=None if dz is None else dz.cuda(), seq_offsets=None if off is None else off.cuda(),
                             score=code(score), before=None if before is None else before.cuda())
    torch.cuda.synchronize()
    L = l.double().numpy()
    n64 = lambda v: None if v is None else v.double().numpy()   # noqa: E731
    ref = ob.balance_loss_backward(L, counts, n64(dl), k, n64(dz), offs, score, n64(before))
    p, lse = ob.probabilities(L, score), ob.log_sum_exp(L)
    ep, el = p_error(L)
    c = ob.clean(L)
    with np.errstate(over="ignore"):
        rest = 1 / (1 + np.exp(c)) if score == "sigmoid" else np.ones_like(c)
        er = (np.minimum(np.abs(c), 200.0) + 4) * 2 * U if score == "sigmoid" else np.zeros_like(c)
    err = np.zeros((T, E))
    for s, (a, b) in enumerate(ob.bounds(offs, T)):
        n = max(b - a, 1)
        gg = np.abs(float(dl[s])) * E / (k * n) * counts[s] / n
        P, e = p[a:b], ep[a:b]
        dot = (P * gg).sum(1, keepdims=True)
        edot = (P * gg * (e + 22 * U)).sum(1, keepdims=True)
        err[a:b] = rest[a:b] * (P * (gg + dot) * (e + er[a:b] + 10 * U) + P * edot)
        if dz is not None:
            f = 2 * abs(float(dz[s])) / n
            err[a:b] += P * f * (np.abs(lse[a:b])[:, None] * (e + 10 * U) + el[a:b][:, None])
    if before is not None:
        err += U * np.abs(n64(before))
    err += 2 * U * np.abs(ref) + TINY
    if l.dtype == BF16:
        err += 2.0 ** -8 * (np.abs(ref) + err)
    worst = np.abs(f64(d) - ref) - err
    assert (worst <= 0).all(), (np.unravel_index(worst.argmax(), worst.shape), float(worst.max()))
    return d


CASES = [(1, 1, 1, 0), (1, 4, 1, 0), (2, 7, 3, 1), (31, 16, 2, 3), (32, 64, 8, 1), (33, 65, 8, 4), (200, 128, 6, 7),
         (1000, 129, 4, 0), (777, 256, 8, 64), (500, 257, 8, 5), (100, 512, 16, 3), (70, 513, 32, 2), (40, 1024, 32, 3),
         (9000, 60, 4, 11)]


@pytest.mark.parametrize("T,E,k,S", CASES)
@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_forward_and_backward(T, E, k, S, kind, score):
    print("CASE balance", T, E, k, S, kind, score, flush=True)
    l, ids, off = inputs(T, E, k, S, kind, T + E)
    check_forward(l, ids, off, score)
    check_backward(l, ids, off, score, T)


def test_without_the_optional_outputs():
    l, ids, off = inputs(100, 40, 4, 5, F32, 3)
    a, b = forward(l, ids, off, "softmax"), forward(l, ids, off, "softmax", z=False, probs=False)
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["counts"], b["counts"])
    check_backward(l, ids, off, "softmax", 1, add=False, z=False)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", [F32, BF16])
def test_masked_and_extreme_logits(score, kind):
    l, ids, off = inputs(64, 24, 3, 4, kind, 5, std=4.0)
    l[0] = -float("inf")                                     # a token without experts
    l[1] = float("nan")
    l[2, ::2] = -float("inf")
    l[3, 5] = float("nan")
    l[4] = torch.finfo(kind).min                             # a mask by the lowest value, all and some
    l[5, 3:] = torch.finfo(kind).min
    l[6] = -90.0                                             # every sigmoid below fp32's normal range
    l[7] = 90.0
    check_forward(l, ids, off, score)
    check_backward(l, ids, off, score, 6)


def test_infinite_logits_are_the_largest_number():
    l, ids, off = inputs(8, 16, 2, 2, F32, 7)
    m = l.clone()
    l[3, 2], m[3, 2] = float("inf"), torch.finfo(F32).max
    for score in ("softmax", "sigmoid"):
        a, b = forward(l, ids, off, score, z=False), forward(m, ids, off, score, z=False)
        assert all(torch.equal(a[n], b[n]) for n in ("loss", "counts", "probs")) and bool(a["probs"].isfinite().all())


def test_sequences_are_independent_and_bits_repeat():
    l, ids, _ = inputs(5000, 96, 8, 0, F32, 8)
    off = torch.tensor([0, 100, 100, 2500, 2501, 5000], dtype=I32)
    a, b = forward(l, ids, off, "softmax"), forward(l, ids, off, "softmax")
    assert all(torch.equal(a[n], b[n]) for n in a)
    assert all((f64(a[n])[1] == 0).all() for n in a)
    m = l.clone()
    m[2500:] = m[2500:].flip(0)
    c = forward(m, ids, off, "softmax")
    assert all(torch.equal(a[n][:3], c[n][:3]) for n in a)


def test_offsets_that_leave_tokens_out_or_are_bad():
    l, ids, _ = inputs(300, 32, 4, 0, F32, 9)
    off = torch.tensor([40, 50, 50, 250], dtype=I32)
    check_forward(l, ids, off, "softmax")
    d = check_backward(l, ids, off, "softmax", 3, add=False)
    assert (f64(d)[:40] == 0).all() and (f64(d)[250:] == 0).all()
    check_forward(l, ids, torch.tensor([-5, 30, 1000], dtype=I32), "softmax")     # read as within [0, T]
    check_backward(l, ids, torch.tensor([-5, 30, 1000], dtype=I32), "softmax", 4)


def test_falling_offsets_write_nothing_else():
    """Results of no meaning, but only where results go."""
    T, E, S = 500, 16, 6
    l, ids, _ = inputs(T, E, 2, 0, F32, 10)
    off = torch.tensor([400, 90, 600, -3, 200, 100, 50], dtype=I32)
    n = mg.balance_loss_workspace_bytes(T, E, S)
    hold = torch.full((n + 512,), SENTINEL, dtype=torch.uint8, device="cuda")
    out = [torch.full((m + 64,), SENTINEL, dtype=torch.uint8, device="cuda") for m in (4 * S, 4 * S, 4 * S * E, 4 * S * E)]
    v = [o[:-64].view(t).view(s) for o, t, s in zip(out, (F32, F32, I32, F32), ((S,), (S,), (S, E), (S, E)))]
    mg.balance_loss(l.cuda(), ids.cuda(), v[0], v[2], hold[:n], probs=v[3], z_loss=v[1], seq_offsets=off.cuda())
    d = torch.full((4 * T * E + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
    mg.balance_loss_backward(l.cuda(), v[2], v[0], d[:-64].view(F32).view(T, E), k=2, seq_offsets=off.cuda())
    torch.cuda.synchronize()
    assert bool((hold[n:] == SENTINEL).all()) and all(bool((o[-64:] == SENTINEL).all()) for o in (*out, d))


def test_before_in_place_and_no_tokens():
    l, ids, off = inputs(90, 33, 3, 4, BF16, 11)
    want = check_backward(l, ids, off, "softmax", 12)
    g = gen(112)
    dl, dz = torch.randn(4, generator=g), torch.randn(4, generator=g)
    d = torch.randn(90, 33, generator=g).to(BF16).cuda()
    counts = torch.from_numpy(ob.balance_loss(l.double().numpy(), ids.numpy(), off.tolist())[2]).to(I32).cuda()
    mg.balance_loss_backward(l.cuda(), counts, dl.cuda(), d, k=3, d_z_loss=dz.cuda(), seq_offsets=off.cuda(), before=d)
    assert torch.equal(d, want)
    e, i = torch.empty(0, 8, device="cuda"), torch.empty(0, 2, dtype=I32, device="cuda")
    loss, counts = buf((1,), F32), buf((1, 8), I32)
    mg.balance_loss(e, i, loss, counts, mg.balance_loss_workspace(0, 8))
    mg.balance_loss_backward(e, counts, loss, e, k=2)
    assert float(loss) == 0 and (counts.cpu() == 0).all()


def test_gradient_by_differences():
    """The gradient's call against differences of the forward call: the loss is off by less than 200 u of itself and z by
    200 u of itself; p's third derivative is below 1, so the loss's below E / (k n^2) max c; (lse^2)''' below 12 (|lse| + 1)."""
    T, E, k, step = 5, 6, 2, 2.0 ** -4
    l, ids, off = inputs(T, E, k, 2, F32, 13)
    off = torch.tensor([0, 3, 5], dtype=I32)
    base = forward(l, ids, off, "softmax")
    dl, dz = torch.tensor([1.0, -2.0]), torch.tensor([0.5, 1.0])
    d = buf((T, E), F32)
    mg.balance_loss_backward(l.cuda(), base["counts"], dl.cuda(), d, k=k, d_z_loss=dz.cuda(), seq_offsets=off.cuda())
    for t, e in [(0, 0), (2, 5), (4, 3)]:
        f, size = [], 0.0
        for sign in (1, -1):
            m = l.clone()
            m[t, e] += sign * step
            o = forward(m, ids, off, "softmax")
            f.append(float((dl.double() * o["loss"].cpu().double() + dz.double() * o["z"].cpu().double()).sum()))
            size = max(size, float((dl.abs() * o["loss"].cpu() + dz.abs() * o["z"].cpu()).sum()))
        s = 0 if t < 3 else 1
        n, lse = (3, 2)[s], float(torch.logsumexp(l[t], 0).abs()) + step
        third = abs(float(dl[s])) * E / (k * n * n) * int(base["counts"][s].max()) + float(dz[s]) / n * 12 * (lse + 1)
        lim = third * step ** 2 / 6 + 200 * U * size / step + 100 * U * (third + 1)
        assert abs((f[0] - f[1]) / (2 * step) - float(d[t, e])) <= lim


def test_graph_and_stream():
    T, E, k, S = 700, 72, 4, 3
    l, d = torch.empty(T, E, device="cuda"), torch.empty(T, E, device="cuda")
    ids, off = torch.empty(T, k, dtype=I32, device="cuda"), torch.empty(S + 1, dtype=I32, device="cuda")
    loss, z, counts, probs = (torch.empty(S, device="cuda"), torch.empty(S, device="cuda"),
                              torch.empty(S, E, dtype=I32, device="cuda"), torch.empty(S, E, device="cuda"))
    ws = mg.balance_loss_workspace(T, E, S)

    def step():
        mg.balance_loss(l, ids, loss, counts, ws, probs=probs, z_loss=z, seq_offsets=off)
        mg.balance_loss_backward(l, counts, loss, d, k=k, d_z_loss=z, seq_offsets=off)

    def fill(seed):
        for v, x in zip((l, ids, off), inputs(T, E, k, S, F32, seed)):
            v.copy_(x)
    outs = (loss, z, counts, probs, d)
    fill(1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    first = [v.clone() for v in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 20, 30, 1):
        fill(seed)
        for v in outs:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [v.clone() for v in outs]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, outs))
    assert all(torch.equal(a, b) for a, b in zip(first, outs))
