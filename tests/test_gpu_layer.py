"""Routing, token permutation and activation checkpoints on MI355X against the fp64 oracle (oracle/layer.py).

Bounds, with u = 2^-24 (half a step of fp32):
- ids, m_sizes and rows: equal.
- routing weights: e^x of a rounded difference x is off by |x| u + 2 u, a sum of E terms in tree order by less than
  16 u, a division and two products by u each: rel <= (|x|max + 24) 2u.  The gradient of the logits adds products and
  a difference: the same relative to the sum of its terms' magnitudes; bf16 adds half a step, 2^-8.
- a sum in fp32: (terms in a lane's chain + steps of the tree) u times the sum of the terms' magnitudes; bf16: 2^-8.
- a scale amax / 448: u for the division plus the error of the amax; a code: half an e4m3 step at v / s (2^-4 of the
  value above 2^-6, 2^-10 below) plus 4 u |v / s| for the reciprocal and products, plus the error of v.
- SwiGLU and its gradient: sigmoid by exp2 and reciprocal is off by (1.5 |g| + 4) 2u relative, each product by u:
  (2 |g| + 8) 2u times the magnitude of the terms.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from oracle import gemm as og
from oracle import layer as ol

pytestmark = pytest.mark.gpu
E4M3, BF16 = torch.float8_e4m3fn, torch.bfloat16
U = 2.0 ** -24
DEC = np.array([og.dec_e4m3(c) for c in range(256)])
SENTINEL = 0x5A


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def buf(shape, dtype):
    """A device buffer full of a sentinel byte."""
    z = torch.empty(0, dtype=dtype).element_size()
    return torch.full((*shape[:-1], shape[-1] * z), SENTINEL, dtype=torch.uint8, device="cuda").view(dtype)


def untouched(t, rows):
    b = t.reshape(-1, t.shape[-1])[rows].view(torch.uint8)
    return bool((b == SENTINEL).all())


def f64(t):
    if t.dtype == E4M3:
        return DEC[t.cpu().view(torch.uint8).numpy()]
    return t.detach().cpu().double().numpy()


def half_step(q):
    """Half an e4m3 step at |q| (a value within 2^-20 of a power of two counts as above it)."""
    e = np.floor(np.log2(np.maximum(np.abs(q) * (1 + 2.0 ** -20), 2.0 ** -6)))
    return np.exp2(e - 4)


def check_codes(codes, s, v, v_err=0.0):
    """codes (decoded) against values v with error v_err, stored with scales s."""
    q = v / s
    lim = half_step(q) + 4 * U * np.abs(q) + v_err / s
    d = np.abs(codes - q)
    assert (d <= lim).all(), float((d / lim).max())


def check_scales(s, v_groups, err_groups, pow2):
    """Scales s against groups of values [..., n] with errors err_groups."""
    amax = np.abs(v_groups).max(axis=-1)
    err = np.max(err_groups, axis=-1) if np.ndim(err_groups) else err_groups
    if pow2:
        lo, hi = ol.scale_of(np.maximum(amax - err, 0) * (1 - U), True), ol.scale_of((amax + err) * (1 + U), True)
        assert ((s == lo) | (s == hi) | (s == ol.scale_of(amax, True))).all()
    else:
        ref = ol.scale_of(amax, False)
        assert (np.abs(s - ref) <= U * ref + 2.0 ** -150 + err / 448).all()


def e8m0(b):
    return np.exp2(b.cpu().numpy().astype(np.float64) - 127)


# ------------------------------------------------------------------ routing

def run_route(logits, k, rows_total, bias=None, score="softmax", stream=None, **kw):
    T, E = logits.shape
    out = dict(ids=buf((T, k), torch.int32), weights=buf((T, k), torch.float32), m_sizes=buf((E,), torch.int32),
               row_of=buf((T, k), torch.int32))
    ws = mg.route_workspace(T, E)
    mg.route(logits, *out.values(), ws, rows_total=rows_total, bias=bias,
             score=mg.SCORE_SIGMOID if score == "sigmoid" else mg.SCORE_SOFTMAX, stream=stream, **kw)
    return out


def check_route(logits, k, rows_total, bias=None, score="softmax", renorm=True, scale=1.0, seg_align=1, cap=0, **kw):
    got = run_route(logits, k, rows_total, bias, score, renorm=renorm, scale=scale, seg_align=seg_align, cap=cap, **kw)
    l = f64(logits)
    ids, w = ol.route(l, k, score, None if bias is None else f64(bias), renorm=renorm, scale=scale, **kw)
    m, row = ol.rows_of(ids, l.shape[1], rows_total, seg_align, cap)
    assert np.array_equal(got["ids"].cpu().numpy(), ids)
    assert np.array_equal(got["m_sizes"].cpu().numpy(), m)
    assert np.array_equal(got["row_of"].cpu().numpy(), row)
    clean = np.where(np.isnan(l), -np.inf, np.minimum(l, ol.FLT_MAX))
    fin = clean[np.isfinite(clean)]
    span = min(float(fin.max() - fin.min()), 110.0) if len(fin) else 0.0
    assert (np.abs(f64(got["weights"]) - w) <= (span + 24) * 2 * U * w + scale * 2.0 ** -125).all()
    return got, ids


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [
    (1, 1, 1, "float32"), (1, 7, 7, "float32"), (3, 64, 8, "bfloat16"), (64, 65, 1, "float32"), (65, 65, 6, "float32"),
    (63, 160, 32, "bfloat16"), (129, 256, 8, "float32"), (300, 300, 4, "bfloat16"), (70, 1000, 9, "float32"),
    (4100, 16, 2, "bfloat16")])
def test_route(T, E, k, dtype, score, renorm):
    l = torch.randn(T, E, generator=gen(T * 7 + E)).to(getattr(torch, dtype)).cuda()
    check_route(l, k, T * k, score=score, renorm=renorm, scale=2.5)


@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,k,n,top,group_top", [
    (5, 8, 2, 8, 3, 1), (33, 8, 2, 8, 3, 2), (100, 256, 8, 8, 4, 2), (70, 96, 5, 2, 1, 2), (66, 592, 6, 16, 3, 1),
    (40, 1024, 8, 64, 10, 2), (17, 111, 4, 3, 3, 2), (200, 512, 16, 4, 2, 2)])
def test_route_groups(T, E, k, n, top, group_top, with_bias):
    g = gen(T + E)
    l = torch.randn(T, E, generator=g).cuda()
    bias = (torch.randn(E, generator=g) * 0.1).cuda() if with_bias else None
    for score in ("softmax", "sigmoid"):
        check_route(l, k, T * k, bias=bias, score=score, n_groups=n, topk_groups=top, group_top=group_top)


def test_route_ties_signed_zeros_and_hollow_rows():
    E = 70
    l = torch.zeros(12, E)
    l[1, ::2] = -0.0                                       # equal to +0: the lowest ids
    l[2] = float("nan")
    l[3] = -float("inf")
    l[4, 3:] = -float("inf")                               # three candidates for five picks
    l[5, [9, 60, 69]] = float("inf")
    l[6] = torch.finfo(torch.float32).min                  # the lowest finite value is an expert like any other
    l[7, 5] = float("nan")
    l[8, 64:] = 1.0
    l[9] = torch.arange(E) * 1e-45                         # subnormals keep their order
    l[10] = torch.linspace(-200, 200, E)
    l[11] = torch.linspace(-900, -700, E)
    for score in ("softmax", "sigmoid"):
        for renorm in (True, False):
            for dtype in (torch.float32, BF16):
                check_route(l.to(dtype).cuda(), 5, 60, score=score, renorm=renorm)
    bias = torch.zeros(E)
    bias[:3] = float("nan")
    bias[3], bias[4], bias[5] = -float("inf"), float("inf"), torch.finfo(torch.float32).min
    check_route(l.cuda(), 5, 60, bias=bias.cuda(), score="sigmoid")
    check_route(l.cuda(), 5, 60, bias=bias.cuda(), n_groups=7, topk_groups=2, group_top=2)
    check_route(l.cuda(), 5, 60, n_groups=7, topk_groups=1, group_top=1)


def test_route_keys_nearer_than_32_bits():
    """score + bias of two experts differ by 2^-50 .. 2^-30: the order is that of 64 bits."""
    T, E = 40, 64
    l = torch.full((T, E), -30.0)
    bias = torch.full((E,), -1.0)
    bias[10], bias[20] = 0.25, 0.25
    l[:, 10] = -20.0
    l[:, 20] = -20.0 + torch.arange(T) * 2.0 ** -16        # sigmoid(-20) = 2e-9: apart by 2^-45 and more
    got, ids = check_route(l.cuda(), 2, 2 * T, bias=bias.cuda(), score="sigmoid")
    assert ids[0].tolist() == [10, 20] and ids[5].tolist() == [20, 10]


@pytest.mark.parametrize("seg_align,cap,rows", [(16, 0, 100000), (128, 0, 100000), (1, 0, 500), (1, 5, 5 * 24),
                                                (1, 1, 24), (1, 7, 40), (1, 0, 0)])
@pytest.mark.parametrize("T", [0, 50, 700])
def test_route_layouts(T, seg_align, cap, rows):
    l = torch.randn(T, 24, generator=gen(3)) + torch.linspace(0, 2, 24)
    check_route(l.cuda(), 3, rows, seg_align=seg_align, cap=cap)


def test_route_long_call_is_deterministic_and_counts_up():
    """More tokens than 256 tiles of one step: ranks run on across steps and tiles."""
    T, E, k = 40001, 32, 4
    l = torch.randn(T, E, generator=gen(11)).cuda()
    a = run_route(l, k, T * k)
    b = run_route(l, k, T * k)
    ids = a["ids"].cpu().numpy()
    for n in a:
        assert torch.equal(a[n], b[n])
    assert np.array_equal(np.bincount(ids.reshape(-1), minlength=E), a["m_sizes"].cpu().numpy())
    order = np.argsort(ids.reshape(-1), kind="stable")     # (expert, token): each token has an expert once
    row = np.empty(T * k, dtype=np.int64)
    row[order] = np.arange(T * k)
    assert np.array_equal(a["row_of"].cpu().numpy().reshape(-1), row)


@pytest.mark.parametrize("T,E,n", [(16, 96, 1), (17, 96, 3), (24, 128, 1), (25, 64, 1), (32, 250, 1), (33, 60, 1), (255, 256, 8), (1024, 40, 1), (1025, 129, 1), (2500, 512, 8),
                                   (3500, 260, 2), (4097, 64, 4)])
def test_route_sizes_around_the_tiles(T, E, n):
    l = torch.randn(T, E, generator=gen(T)).to(BF16).cuda()
    bias = (torch.randn(E, generator=gen(E)) * 0.1).cuda() if E % 64 == 0 else None
    check_route(l, 4, 4 * T + 64 * E, bias=bias, score="sigmoid", n_groups=n, topk_groups=max(1, n // 2),
                group_top=min(2, n), seg_align=16)


@pytest.mark.parametrize("E", [64, 128, 160, 256, 384, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_route_rows_off_any_wider_alignment(E, dtype):
    """Logits that begin one element into their storage; so do the gradient's."""
    T, k = 20, 6
    back = torch.randn(1 + T * E, generator=gen(E)).to(dtype).cuda()
    l = back[1:].view(T, E)
    _, ids = check_route(l, k, T * k)
    dw = torch.randn(T, k, generator=gen(5))
    ids = torch.tensor(ids, dtype=torch.int32).cuda()
    a, b = torch.full((2 + T * E,), 7.0, dtype=dtype, device="cuda"), buf((T, E), dtype)
    for renorm in (True, False):
        mg.route_backward(l, ids, dw.cuda(), a[1:-1].view(T, E), renorm=renorm)
        mg.route_backward(l.clone(), ids, dw.cuda(), b, renorm=renorm)
        assert torch.equal(a[1:-1].view(T, E), b) and a[0] == 7 and a[-1] == 7


@pytest.mark.parametrize("T,E,k", [(70001, 24, 3), (65535, 9, 2), (65536, 9, 2)])
def test_route_rows_past_16_bit_counts(T, E, k):
    """An expert's assignments below and above 2^16."""
    l = torch.randn(T, E, generator=gen(T))
    l[:, 3] += 20                                          # every token's first choice
    got = run_route(l.cuda(), k, T * k)
    ids = got["ids"].cpu().numpy()
    m, row = ol.rows_of(ids, E, T * k, 1, 0)
    assert (ids[:, 0] == 3).all() and m[3] == T
    assert np.array_equal(got["m_sizes"].cpu().numpy(), m) and np.array_equal(got["row_of"].cpu().numpy(), row)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k,dtype", [(1, 1, 1, "float32"), (5, 64, 8, "float32"), (33, 160, 6, "bfloat16"),
                                         (3, 300, 32, "float32"), (9, 1000, 4, "bfloat16"), (130, 7, 7, "float32")])
def test_route_backward(T, E, k, dtype, score, renorm):
    g = gen(T + E + k)
    l = torch.randn(T, E, generator=g).to(getattr(torch, dtype))
    ids = torch.argsort(l.float(), dim=1, descending=True)[:, :k].to(torch.int32)
    ids[T // 2, k - 1] = -1
    if T > 4:
        ids[0] = -1
        l[1, 0] = -float("inf")
        ids[1, 0] = 0                                      # a chosen expert whose score is 0
    dw = torch.randn(T, k, generator=g)
    d = buf((T, E), l.dtype)
    mg.route_backward(l.cuda(), ids.cuda(), dw.cuda(), d, renorm=renorm, scale=2.5,
                      score=mg.SCORE_SIGMOID if score == "sigmoid" else mg.SCORE_SOFTMAX)
    x, i, w = f64(l), ids.numpy(), f64(dw)
    ref = ol.route_backward(x, i, w, score, renorm, 2.5)
    s = ol.scores(x, score)
    span = float((x[np.isfinite(x)].max() - x[np.isfinite(x)].min()))
    chosen = np.zeros((T, E))
    wsum = np.zeros((T, 1))
    for t in range(T):
        at = [j for j in range(k) if i[t, j] >= 0]
        z = s[t, i[t, at]].sum() if renorm else 1.0
        z = z if z > 0 else 1.0
        wsum[t] = (np.abs(w[t, at]) * s[t, i[t, at]] / z).sum()
        for j in at:
            chosen[t, i[t, j]] = np.abs(w[t, j])
    if renorm:                                             # only the chosen experts' logits have gradients
        zs = np.array([max(s[t, [e for e in i[t] if e >= 0]].sum(), 1e-300) for t in range(T)])[:, None]
        mag = np.where(chosen > 0, 2.5 * s / zs * (chosen + wsum), 0)
    elif score == "softmax":
        mag = 2.5 * s * (chosen + wsum)
    else:
        mag = 2.5 * s * chosen
    lim = (span + 40) * 2 * U * mag + 2.0 ** -125 + (2.0 ** -8 * np.abs(ref) if dtype == "bfloat16" else 0)
    err = np.abs(f64(d) - ref)
    assert (err <= lim).all(), float((err / lim).max())


# ------------------------------------------------------------------ permutation

def some_rows(T, k, rows, seed, bad=True):
    """row_of [T, k]: distinct rows, some assignments without one, some values out of range."""
    g = gen(seed)
    n = min(T * k, rows)
    flat = torch.full((T * k,), -1, dtype=torch.int64)
    flat[torch.randperm(T * k, generator=g)[:n]] = torch.randperm(rows, generator=g)[:n]
    if bad and T * k > 4:
        flat[torch.randperm(T * k, generator=g)[:T * k // 5]] = -1
        flat[0], flat[-1] = rows, 2 ** 31 - 1
        flat[T * k // 2] = -(2 ** 31)
    return flat.reshape(T, k).to(torch.int32)


def check_rows_operand(A, A_scale, values, fmt, rows):
    """Rows of an operand in its format against {row: fp64 values with error 0 (bf16: exactly rounded)}."""
    width = A.shape[-1]
    free = [r for r in range(rows) if r not in values]
    assert untouched(A, free)
    at = sorted(values)
    if not at:
        return
    v = np.stack([values[r] for r in at])
    got = f64(A.reshape(rows, width)[at])
    if fmt == "bf16":
        assert (np.abs(got - v) <= 2.0 ** -8 * np.abs(v) + U * np.abs(v)).all()
        return
    sc = A_scale.reshape(rows, -1) if fmt == "rows" else A_scale.t()
    assert untouched(sc.contiguous(), free)
    s = e8m0(sc[at]) if fmt == "e8m0" else f64(sc[at])
    grp = v.reshape(len(at), -1, 128)
    check_scales(s, grp, U * np.abs(grp).max(-1, keepdims=True), fmt == "e8m0")
    check_codes(got, np.repeat(s, 128, axis=1), v, U * np.abs(v))


def operand(lead, rows, width, fmt):
    if fmt == "bf16":
        return buf((*lead, width), BF16), None
    if fmt == "rows":
        return buf((*lead, width), E4M3), buf((*lead, width // 128), torch.float32)
    return buf((*lead, width), E4M3), buf((width // 128, rows), torch.float32 if fmt == "km" else torch.uint8)


PERMUTE = [(1, 1, 128, 1), (1, 8, 1152, 40), (5, 3, 256, 12), (37, 9, 1024, 300), (96, 8, 2176, 500), (300, 2, 7168, 600)]


@pytest.mark.parametrize("fmt", ["bf16", "rows", "km", "e8m0"])
@pytest.mark.parametrize("T,k,K,rows", PERMUTE)
def test_dispatch(T, k, K, rows, fmt):
    x = torch.randn(T, K, generator=gen(T + K)).to(BF16)
    x[0, :128] = 0                                         # a group of zeros: scale 1
    if K >= 512:
        x[0, 128:256] *= 1e-38                             # scales below the smallest normal number
        x[0, 256:384] = 1e-40
        x[0, 384:512] *= 1e36
    row_of = some_rows(T, k, rows, 5)
    A, sc = operand((rows,), rows, K, fmt)
    mg.dispatch(x.cuda(), row_of.cuda(), A, sc, scale_km=fmt == "km")
    vals = ol.dispatch(f64(x), row_of.numpy(), rows)
    if fmt == "bf16":
        got = A.cpu()
        for r, v in vals.items():
            assert np.array_equal(f64(got[r]), v)
    check_rows_operand(A, sc, vals, fmt, rows)


@pytest.mark.parametrize("K", [1, 2, 7, 9, 513, 1023, 2050])
def test_dispatch_and_combine_odd_widths(K):
    T, k, rows = 33, 3, 90
    x = torch.randn(T, K, generator=gen(K)).to(BF16)
    row_of = some_rows(T, k, rows, 6)
    back = torch.zeros(1 + rows * K, dtype=BF16, device="cuda")
    A = back[1:].view(rows, K)                             # 2-byte aligned
    mg.dispatch(x.cuda(), row_of.cuda(), A)
    for r, v in ol.dispatch(f64(x), row_of.numpy(), rows).items():
        assert np.array_equal(f64(A[r]), v)
    w = torch.rand(T, k, generator=gen(1))
    out = buf((T, K), BF16)
    mg.combine(A, row_of.cuda(), out, w.cuda())
    ref, mag = ol.combine(f64(A), row_of.numpy(), f64(w), rows)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * (k + 1) * U * mag).all()
    dY, dw = buf((rows, K), BF16), buf((T, k), torch.float32)
    mg.combine_backward(x.cuda(), A, w.cuda(), row_of.cuda(), dY, dw)
    rY, rw, magw = ol.combine_backward(f64(x), f64(A), f64(w), row_of.numpy(), rows)
    check_rows_operand(dY, None, rY, "bf16", rows)
    assert (np.abs(f64(dw) - rw) <= (8 * -(-K // 2048) + 24) * U * magw).all()


@pytest.mark.parametrize("fmt", ["rows", "km"])
def test_dispatch_codes_on_rounding_borders(fmt):
    """bf16 values over a bf16 maximum lie on e4m3's borders once in two hundred: codes are those of the fp32 quotient."""
    T, K, k = 64, 1024, 2
    x = torch.randn(T, K, generator=gen(21)).to(BF16)
    g = x.float().reshape(T, -1, 128)
    s = g.abs().amax(-1) / 448
    q = g / s[..., None]
    ratio = g.double() / s.double()[..., None]
    near = torch.frexp(ratio)[0].abs() * 16 % 1            # a border has 4 bits after the leading one, the last set
    assert ((near - 0.5).abs() < 2.0 ** -19).sum() > 200   # there are such values here
    A, sc = operand((T * k,), T * k, K, fmt)
    mg.dispatch(x.cuda(), torch.arange(T * k, dtype=torch.int32).view(T, k).cuda(), A, sc, scale_km=fmt == "km")
    want = q.clamp(-448, 448).to(E4M3).reshape(T, K).view(torch.uint8).repeat_interleave(k, 0)
    assert torch.equal(A.cpu().view(torch.uint8), want)
    assert torch.equal((sc.t() if fmt == "km" else sc).cpu(), s.repeat_interleave(k, 0))


def test_dispatch_special_values():
    K = 512
    x = torch.randn(2, K, generator=gen(2)).to(BF16)
    x[0, 5], x[0, 130], x[1, 300] = float("nan"), float("inf"), -float("inf")
    row_of = torch.tensor([[0], [1]], dtype=torch.int32)
    for fmt in ("rows", "e8m0"):
        A, sc = operand((4,), 4, K, fmt)
        mg.dispatch(x.cuda(), row_of.cuda(), A, sc)
        codes = A.cpu().view(torch.uint8).numpy()
        s = f64(sc)[:2] if fmt == "rows" else sc.cpu().numpy().T[:2].astype(np.float64)
        assert codes[0, 5] & 0x7F == 0x7F                  # NaN stays, and does not count for the scale
        ref = np.abs(np.delete(f64(x)[0, :128], 5)).max() / 448
        assert abs((s[0, 0] if fmt == "rows" else ref) - ref) <= U * ref
        inf = np.isinf(s) if fmt == "rows" else s == 255
        assert inf.tolist() == [[False, True, False, False], [False, False, True, False]]
        assert codes[0, 130] & 0x7F == 0x7F and (np.delete(codes[0, 128:256], 2) & 0x7F == 0).all()


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("T,k,N,rows", PERMUTE)
def test_combine(T, k, N, rows, weighted):
    Y = torch.randn(rows, N, generator=gen(N)).to(BF16)
    row_of = some_rows(T, k, rows, 7)
    row_of[T // 2] = -1                                    # a token without any row: 0
    free = sorted(set(range(rows)) - {int(r) for r in row_of.reshape(-1)})
    Y[free] = float("nan")                                 # rows that no token has are not read
    w = torch.rand(T, k, generator=gen(1)) if weighted else None
    out = buf((T, N), BF16)
    mg.combine(Y.cuda(), row_of.cuda(), out, None if w is None else w.cuda())
    Y[free] = 0
    ref, mag = ol.combine(f64(Y), row_of.numpy(), None if w is None else f64(w), rows)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * (k + 1) * U * mag).all()


@pytest.mark.parametrize("fmt", ["bf16", "rows", "km", "e8m0"])
@pytest.mark.parametrize("T,k,N,rows", PERMUTE)
def test_combine_backward(T, k, N, rows, fmt):
    g = gen(N + T)
    dout, Y, w = torch.randn(T, N, generator=g).to(BF16), torch.randn(rows, N, generator=g).to(BF16), torch.rand(T, k, generator=g)
    w[0, 0] = 0
    row_of = some_rows(T, k, rows, 8)
    dY, sc = operand((rows,), rows, N, fmt)
    dw = buf((T, k), torch.float32)
    mg.combine_backward(dout.cuda(), Y.cuda(), w.cuda(), row_of.cuda(), dY, dw, sc, scale_km=fmt == "km")
    rY, rw, mag = ol.combine_backward(f64(dout), f64(Y), f64(w), row_of.numpy(), rows)
    check_rows_operand(dY, sc, rY, fmt, rows)
    assert (np.abs(f64(dw) - rw) <= (8 * -(-N // 2048) + 24) * U * mag).all()


def test_capacity_buffers():
    """[G, cap, K] operands take the rows e * cap + r that routing gives them, and overflow is dropped."""
    T, E, k, K, cap = 50, 6, 2, 256, 9
    l = torch.randn(T, E, generator=gen(4)).cuda()
    r = run_route(l, k, E * cap, cap=cap)
    x = torch.randn(T, K, generator=gen(5)).to(BF16)
    assert int(r["m_sizes"].max()) > cap                    # some are dropped
    vals = ol.dispatch(f64(x), r["row_of"].cpu().numpy(), E * cap)
    for fmt in ("bf16", "rows", "km"):
        A, sc = operand((E, cap), E * cap, K, fmt)
        mg.dispatch(x.cuda(), r["row_of"], A, sc, scale_km=fmt == "km")
        check_rows_operand(A, sc, vals, fmt, E * cap)
    Y, out = torch.randn(E, cap, K, generator=gen(6)).to(BF16), buf((T, K), BF16)
    mg.combine(Y.cuda(), r["row_of"], out, r["weights"])
    ref, mag = ol.combine(f64(Y).reshape(-1, K), r["row_of"].cpu().numpy(), f64(r["weights"]), E * cap)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * (k + 1) * U * mag).all()


def test_offsets_past_32_bits():
    """Rows whose byte offset is past 2^32 (bf16 and e4m3), and whose element offset is past 2^31."""
    K, rows, T = 7168, 700_000, 6
    row_of = torch.tensor([[0], [299_600], [299_700], [599_186], [599_187], [rows - 1]], dtype=torch.int32)
    x = torch.randn(T, K, generator=gen(8)).to(BF16)
    A = torch.empty(rows, K, dtype=BF16, device="cuda")
    mg.dispatch(x.cuda(), row_of.cuda(), A)
    assert torch.equal(A[row_of.reshape(-1).long().cuda()].cpu(), x)
    out = buf((T, K), BF16)
    mg.combine(A, row_of.cuda(), out)
    assert torch.equal(out.cpu(), x)
    Q, sc = A.view(-1)[:rows * K // 2].view(torch.uint8).view(rows, K).view(E4M3), torch.empty(rows, K // 128, device="cuda")
    mg.dispatch(x.cuda(), row_of.cuda(), Q, sc)
    at = row_of.reshape(-1).long().cuda()
    check_codes(f64(Q.view(torch.uint8)[at].view(E4M3)), np.repeat(f64(sc[at]), 128, axis=1), f64(x))


# ------------------------------------------------------------------ checkpoints

COUNTS = [([1], 1), ([128], 128), ([129, 0, 127, 1, 300], 557), ([0, 0, 5], 9), ([40, -3, 20], 60),
          ([100, 200, 50], 270), ([0], 3), ([3, 0, 140, 64] * 20, 4140)]
# (counts, rows of the buffers): short and empty segments, rows of nobody, a negative count, segments past the end


def used_rows(counts, rows):
    return min(sum(max(c, 0) for c in counts), rows)


def gate_up(rows, I, seed):
    gu = torch.randn(rows, 2 * I, generator=gen(seed))
    gu[0, :32] = torch.linspace(-100, 100, 32)             # gates whose sigmoid saturates
    if rows > 1:
        gu[1] = 0
    return gu


@pytest.mark.parametrize("fmt", ["bf16", "rows", "km"])
@pytest.mark.parametrize("I", [128, 640])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_swiglu_checkpoint(counts, rows, I, fmt):
    n = used_rows(counts, rows)
    gu = gate_up(rows, I, rows + I).to(BF16)
    gu[n:] = float("nan")
    H, hs = operand((rows,), rows, I, fmt)
    ck, cs = operand((rows,), rows, 2 * I, "rows")
    mg.swiglu_checkpoint(gu.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), H, ck, cs, hs, scale_km=fmt == "km")
    tail = list(range(n, rows))
    assert untouched(H, tail) and untouched(ck, tail) and untouched(cs, tail)
    if hs is not None:
        assert untouched((hs.t() if fmt == "km" else hs).contiguous(), tail)
    if n == 0:
        return
    v = f64(gu[:n])
    s = f64(cs[:n])
    check_scales(s, v.reshape(n, -1, 128), 0.0, False)
    check_codes(f64(ck[:n]), np.repeat(s, 128, axis=1), v)
    h, (g, _) = ol.swiglu(v), ol.split_gate_up(v)
    err = (2 * np.abs(g) + 8) * 2 * U * np.abs(h)
    if fmt == "bf16":
        assert (np.abs(f64(H[:n]) - h) <= 2.0 ** -8 * (np.abs(h) + err) + err + 1e-36).all()
        return
    s = f64(hs.t()[:n] if fmt == "km" else hs[:n])
    check_scales(s, h.reshape(n, -1, 128), (err + 1e-36).reshape(n, -1, 128), False)
    check_codes(f64(H[:n]), np.repeat(s, 128, axis=1), h, err + 1e-36)


def checkpoint(rows, I, seed, counts):
    """A checkpoint and dH with NaN in the rows of nobody."""
    gu = gate_up(rows, I, seed)
    s = ol.row_scales(gu.double().numpy())
    s32 = torch.tensor(s, dtype=torch.float32)
    codes = (gu / s32.repeat_interleave(128, 1)).clamp(-448, 448).to(E4M3)
    dh = (torch.randn(rows, I, generator=gen(seed + 1)) * 0.02).to(BF16)
    n = used_rows(counts, rows)
    s32[n:], dh[n:] = float("nan"), float("nan")
    v = f64(codes[:n]) * np.repeat(f64(s32[:n]), 128, axis=1)
    d, h = ol.swiglu_backward(v, f64(dh[:n]))
    g, u = ol.split_gate_up(v)
    sg = ol.sigmoid(g)
    rel = (2 * np.abs(g) + 10) * 2 * U
    d_err = ol.interleave(np.abs(f64(dh[:n]) * u) * (sg + np.abs(g) * sg) * rel, np.abs(f64(dh[:n]) * g * sg) * rel) + 1e-36
    return codes, s32, dh, n, d, d_err, h, np.abs(h) * rel + 1e-36


@pytest.mark.parametrize("I", [128, 640])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_swiglu_checkpoint_backward(counts, rows, I):
    ck, cs, dh, n, d, d_err, h, h_err = checkpoint(rows, I, 3, counts)
    dGU, H = buf((rows, 2 * I), BF16), buf((rows, I), BF16)
    mg.swiglu_checkpoint_backward(dh.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), ck.cuda(), cs.cuda(), dGU, H)
    tail = list(range(n, rows))
    assert untouched(dGU, tail) and untouched(H, tail)
    assert (np.abs(f64(dGU[:n]) - d) <= 2.0 ** -8 * np.abs(d) + 1.01 * d_err).all()
    assert (np.abs(f64(H[:n]) - h) <= 2.0 ** -8 * np.abs(h) + 1.01 * h_err).all()


def check_token_groups(X_k, X_k_scale, v, err, counts, rows, e8):
    """Codes and scales of token groups against values v [n, M]."""
    groups = ol.token_groups(counts, rows)
    S = X_k_scale.shape[0]
    assert untouched(X_k_scale, list(range(min(len(groups), S), S)))
    assert untouched(X_k, list(range(v.shape[0], rows)))
    codes = f64(X_k[:v.shape[0]])
    s = e8m0(X_k_scale) if e8 else f64(X_k_scale)
    for i, (a, b) in enumerate(groups):
        if i >= S:
            continue
        check_scales(s[i], v[a:b].T, err[a:b].T, e8)
        check_codes(codes[a:b], s[i][None, :], v[a:b], err[a:b])


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("fmt", ["rows", "km"])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_swiglu_checkpoint_backward_fp8(counts, rows, fmt, e8):
    for I in (128, 384):
        ck, cs, dh, n, d, d_err, h, h_err = checkpoint(rows, I, 4, counts)
        S = mg.k_scale_groups(counts) + 2
        dGU, ds = operand((rows,), rows, 2 * I, fmt)
        kdt = torch.uint8 if e8 else torch.float32
        dk, dks, hk, hks = buf((rows, 2 * I), E4M3), buf((S, 2 * I), kdt), buf((rows, I), E4M3), buf((S, I), kdt)
        mg.swiglu_checkpoint_backward_fp8(dh.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), ck.cuda(), cs.cuda(),
                                          dGU, ds, dk, dks, hk, hks, scale_km=fmt == "km")
        tail = list(range(n, rows))
        sc = (ds.t() if fmt == "km" else ds).contiguous()
        assert untouched(dGU, tail) and untouched(sc, tail)
        if n:
            s = f64(sc[:n])
            check_scales(s, d.reshape(n, -1, 128), d_err.reshape(n, -1, 128), False)
            check_codes(f64(dGU[:n]), np.repeat(s, 128, axis=1), d, d_err)
        check_token_groups(dk, dks, d, d_err, counts, rows, e8)
        check_token_groups(hk, hks, h, h_err, counts, rows, e8)


@pytest.mark.parametrize("e8", [False, True])
@pytest.mark.parametrize("src", ["bf16", "rows", "km"])
@pytest.mark.parametrize("counts,rows", COUNTS)
def test_checkpoint_to_k_groups(counts, rows, src, e8):
    M, n = 512, used_rows(counts, rows)
    x = torch.randn(rows, M, generator=gen(rows))
    x[:, 7] = 0                                            # a column of zeros: scale 1
    x[:, 300] *= 1e-38                                     # and of tiny values
    if src == "bf16":
        X, sc = x.to(BF16), None
        X[n:] = float("nan")
        v = f64(X[:n])
    else:
        sc = torch.tensor(ol.row_scales(x.double().numpy()), dtype=torch.float32)
        X = (x / sc.repeat_interleave(128, 1)).to(E4M3)
        sc[n:] = float("nan")
        v = f64(X[:n]) * np.repeat(f64(sc[:n]), 128, axis=1)
    S = mg.k_scale_groups(counts) + 1
    X_k, ks = buf((rows, M), E4M3), buf((S, M), torch.uint8 if e8 else torch.float32)
    mg.checkpoint_to_k_groups(X.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), X_k, ks,
                              None if sc is None else (sc.t().contiguous() if src == "km" else sc).cuda(),
                              scale_km=src == "km")
    check_token_groups(X_k, ks, v, U * np.abs(v) + 2.0 ** -149, counts, rows, e8)


def test_fewer_scale_groups_than_the_histogram_needs():
    counts, rows, M = [200, 10, 128], 338, 256
    x = torch.randn(rows, M, generator=gen(1)).to(BF16)
    back = buf((4, M), torch.float32)
    X_k = buf((rows, M), E4M3)
    mg.checkpoint_to_k_groups(x.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), X_k, back[:2])
    assert untouched(back, [2, 3]) and not untouched(back, [0, 1])
    check_token_groups(X_k, back[:2], f64(x), U * np.abs(f64(x)), counts, rows, False)


def test_many_experts_token_groups():
    """More experts than a wave has lanes, most of them empty or short."""
    rng = np.random.default_rng(3)
    counts = [int(c) for c in rng.integers(0, 4, 700)]
    counts[650] = 300
    rows, M = sum(counts), 256
    x = torch.randn(rows, M, generator=gen(2)).to(BF16)
    X_k, ks = buf((rows, M), E4M3), buf((mg.k_scale_groups(counts), M), torch.float32)
    mg.checkpoint_to_k_groups(x.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), X_k, ks)
    check_token_groups(X_k, ks, f64(x), U * np.abs(f64(x)), counts, rows, False)


def test_checkpoint_offsets_past_32_bits():
    """The last rows of buffers of 4 to 9 GB come out as a call on those rows alone computes them, bit for bit."""
    rows, tail, I = 540_000, 300, 4096
    counts = [rows - tail, 0, tail]
    m, m_tail = (torch.tensor(c, dtype=torch.int32).cuda() for c in (counts, [tail]))
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    last = slice(rows - tail, rows)

    def same(a, b):
        assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))

    def forward(gu, m_sizes):
        n = gu.shape[0]
        H, hs = operand((n,), n, I, "km")
        ck, cs = operand((n,), n, 2 * I, "rows")
        mg.swiglu_checkpoint(gu, m_sizes, H, ck, cs, hs, scale_km=True)
        return H, hs, ck, cs

    def backward(dh, m_sizes, ck, cs):
        n, S = dh.shape[0], mg.k_scale_groups(m_sizes.tolist())
        dGU, ds = operand((n,), n, 2 * I, "km")
        dk, dks, hk, hks = buf((n, 2 * I), E4M3), buf((S, 2 * I), torch.float32), buf((n, I), E4M3), buf((S, I), torch.float32)
        mg.swiglu_checkpoint_backward_fp8(dh, m_sizes, ck, cs, dGU, ds, dk, dks, hk, hks, scale_km=True)
        return dGU, ds, dk, dks, hk, hks

    gu = torch.empty(rows, 2 * I, dtype=BF16, device="cuda").normal_(generator=g)
    H, hs, ck, cs = forward(gu, m)
    h, hs1, c, cs1 = forward(gu[last].contiguous(), m_tail)
    same(H[last], h), same(hs[:, last], hs1), same(ck[last], c), same(cs[last], cs1)
    del gu, H, hs, h, hs1
    dh = torch.empty(rows, I, dtype=BF16, device="cuda").normal_(generator=g)
    big, small = backward(dh, m, ck, cs), backward(dh[last].contiguous(), m_tail, c, cs1)
    groups = small[3].shape[0]
    for i in (0, 2, 4):
        same(big[i][last], small[i])
    same(big[1][:, last], small[1]), same(big[3][-groups:], small[3]), same(big[5][-groups:], small[5])
    del big, small
    dGU, H2 = buf((rows, 2 * I), BF16), buf((rows, I), BF16)
    d1, h1 = buf((tail, 2 * I), BF16), buf((tail, I), BF16)
    mg.swiglu_checkpoint_backward(dh, m, ck, cs, dGU, H2)
    mg.swiglu_checkpoint_backward(dh[last].contiguous(), m_tail, c, cs1, d1, h1)
    same(dGU[last], d1), same(H2[last], h1)
    X_k, ks, x1, k1 = buf((rows, 2 * I), E4M3), buf((mg.k_scale_groups(counts), 2 * I), torch.uint8), buf((tail, 2 * I), E4M3), \
        buf((groups, 2 * I), torch.uint8)
    mg.checkpoint_to_k_groups(dGU, m, X_k, ks)
    mg.checkpoint_to_k_groups(d1, m_tail, x1, k1)
    same(X_k[last], x1), same(ks[-groups:], k1)


# ------------------------------------------------------------------ streams, graphs

def layer_step(s, stream=None):
    mg.route(s["logits"], s["ids"], s["weights"], s["m_sizes"], s["row_of"], s["ws"], rows_total=s["rows"], stream=stream)
    mg.dispatch(s["x"], s["row_of"], s["A"], s["A_scale"], stream=stream)
    mg.combine(s["Y"], s["row_of"], s["out"], s["weights"], stream=stream)
    mg.combine_backward(s["dout"], s["Y"], s["weights"], s["row_of"], s["dY"], s["d_weights"], stream=stream)
    mg.route_backward(s["logits"], s["ids"], s["d_weights"], s["d_logits"], stream=stream)
    mg.swiglu_checkpoint(s["dY"], s["m_sizes"], s["H"], s["ckpt"], s["ckpt_scale"], stream=stream)
    mg.swiglu_checkpoint_backward_fp8(s["H"], s["m_sizes"], s["ckpt"], s["ckpt_scale"], s["g"], s["g_scale"], s["gk"],
                                      s["gk_scale"], s["hk"], s["hk_scale"], stream=stream)


def layer_state(T, E, k, W, seed):
    g, R = gen(seed), T * k
    S = R // 128 + E
    z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")   # noqa: E731
    q = lambda *shape: z(*shape, dtype=torch.uint8).view(E4M3)                                # noqa: E731
    return dict(rows=R, logits=torch.randn(T, E, generator=g).cuda(), x=torch.randn(T, W, generator=g).to(BF16).cuda(),
                Y=torch.randn(R, W, generator=g).to(BF16).cuda(), dout=torch.randn(T, W, generator=g).to(BF16).cuda(),
                ids=z(T, k, dtype=torch.int32), weights=z(T, k), m_sizes=z(E, dtype=torch.int32),
                row_of=z(T, k, dtype=torch.int32), ws=mg.route_workspace(T, E), A=q(R, W), A_scale=z(R, W // 128),
                out=z(T, W, dtype=BF16), dY=z(R, W, dtype=BF16), d_weights=z(T, k), d_logits=z(T, E),
                H=z(R, W // 2, dtype=BF16), ckpt=q(R, W), ckpt_scale=z(R, W // 128), g=q(R, W), g_scale=z(R, W // 128),
                gk=q(R, W), gk_scale=z(S, W), hk=q(R, W // 2), hk_scale=z(S, W // 2))


def snapshot(s):
    return {n: v.clone().view(torch.uint8) if v.dtype == E4M3 else v.clone() for n, v in s.items()
            if isinstance(v, torch.Tensor) and n != "ws"}


@pytest.mark.parametrize("T", [20, 500])
def test_graph_replays(T):
    """A captured layer follows its inputs, replay after replay, with eager work in between."""
    s = layer_state(T, 16, 2, 512, 1)
    layer_step(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer_step(s)
    for r in range(4):
        other = layer_state(T, 16, 2, 512, 10 + r)
        layer_step(other)
        want = snapshot(other)
        for n in ("logits", "x", "Y", "dout"):
            s[n].copy_(other[n])
        graph.replay()
        torch.cuda.synchronize()
        got = snapshot(s)
        for n in want:
            if n.endswith("k_scale"):                      # rows past this histogram's groups are older ones
                groups = mg.k_scale_groups(s["m_sizes"].tolist())
                assert torch.equal(got[n][:groups], want[n][:groups]), (r, n)
            else:
                assert torch.equal(got[n], want[n]), (r, n)


def test_another_stream():
    s, want = layer_state(300, 16, 2, 512, 2), layer_state(300, 16, 2, 512, 2)
    layer_step(want)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    layer_step(s, stream=st)
    st.synchronize()
    a, b = snapshot(s), snapshot(want)
    for n in a:
        assert torch.equal(a[n], b[n]), n


def test_native_tensor_checks():
    f = mg._args_module().pointers
    x = torch.zeros(3, 4, device="cuda")
    y = torch.zeros(5, dtype=torch.int32, device="cuda")
    e = torch.zeros(0, 4, device="cuda")
    good = (x, "x", (3, 4), torch.float32)
    assert f((good, mg._ABSENT, (y, "y", (5,), torch.int32))) == (x.data_ptr(), None, y.data_ptr())
    assert f(((x, "x", x.shape, x.dtype),)) == (x.data_ptr(),)       # torch.Size is a tuple
    assert f(((e, "e", (0, 4), torch.float32),)) == (e.data_ptr(),)
    for bad in [(x, "x", (3, 5), torch.float32), (x, "x", (3,), torch.float32), (x, "x", (3, 4, 1), torch.float32),
                (x, "x", (3, 4), torch.int32), (x, "x", (3, 2 ** 64 + 4), torch.float32), (x, "x", (3, 4.0), torch.float32),
                (x.t(), "x", (4, 3), torch.float32), (x[:, :2], "x", (3, 2), torch.float32), (x.cpu(), "x", (3, 4), torch.float32)]:
        assert f((bad,)) is None and f((good, bad)) is None and f((bad, good)) is None
