"""RMS norm and its backward pass on MI355X against the fp64 oracle (oracle/block.py).

Bounds, with u = 2^-24 (half a step of fp32); half a step of bf16 is 2^-8 of a value.
- a sum over a row: at most 32 terms in a lane's chain (squares of bf16 are exact), 6 steps in the wave, 16 waves: 54 u
  of the terms' magnitudes.  rstd has half of that, a division, a sum and the root: 27 + 1 + 3 < 32 u relative.
- h rstd weight: two products more, 34 u, then the format's rounding.
- dx: g = dy w and xhat = h rstd are off by u each, their products' mean by (54 + 4) u of the mean magnitude; then three
  fp32 roundings.
- d_weight: xhat is off by u, the product fused; rows in a workgroup's chain, then partial rows in 16 chains and their
  sum: (ceil(T / 256) + 16 + 16 + 2) u of the terms' magnitudes.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from oracle import block as ob
from tests.test_gpu_layer import SENTINEL, U, buf, check_codes, check_scales, e8m0, f64, gen

pytestmark = pytest.mark.gpu
E4M3, BF16, F32 = torch.float8_e4m3fn, torch.bfloat16, torch.float32
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def tokens(T, K, seed):
    g = gen(seed)
    return (torch.randn(T, K, generator=g) * torch.exp(0.7 * torch.randn(K, generator=g)) *
            torch.exp(torch.randn(T, 1, generator=g))).to(BF16)


def weight_of(K, kind, seed):
    return (1 + 0.3 * torch.randn(K, generator=gen(seed))).to(kind)


def outputs(T, K, fmt):
    if fmt == "rows":
        return buf((T, K), E4M3), buf((T, K // 128), F32)
    if fmt == "km":
        return buf((T, K), E4M3), buf((K // 128, T), F32)
    return buf((T, K), E4M3), buf((K // 128, T), torch.uint8)


def check_forward(x, r, w, eps, with_y=True, fmt=None, sum_out=True, stream=None):
    T, K = x.shape
    h = x if r is None else (x.float() + r.float()).to(BF16)
    v, rstd = ob.rms_norm(h.double().numpy(), w.double().numpy(), eps)
    y = buf((T, K), BF16) if with_y else None
    q, qs = outputs(T, K, fmt) if fmt else (None, None)
    so = buf((T, K), BF16) if r is not None and sum_out else None
    rs = buf((T,), F32)
    mg.rms_norm(x.cuda(), w.cuda(), residual=None if r is None else r.cuda(), sum_out=so, y=y, q=q, q_scale=qs, rstd=rs,
                eps=eps, scale_km=fmt == "km", stream=stream)
    torch.cuda.synchronize()
    assert (np.abs(f64(rs) - rstd) <= 32 * U * rstd).all()
    if so is not None:
        assert torch.equal(so.cpu().view(torch.int16), h.view(torch.int16))
    if y is not None:
        assert (np.abs(f64(y) - v) <= (HALF + 34 * U) * np.abs(v) + 2.0 ** -133).all()
    if fmt:
        err = 34 * U * np.abs(v)
        s = e8m0(qs).T if fmt == "e8m0" else (f64(qs).T if fmt == "km" else f64(qs))
        check_scales(s, v.reshape(T, -1, 128), err.reshape(T, -1, 128), fmt == "e8m0")
        check_codes(f64(q).reshape(T, -1, 128), s[..., None], v.reshape(T, -1, 128), err.reshape(T, -1, 128))


@pytest.mark.parametrize("T,K", [(1, 1), (1, 2), (3, 7), (2, 8), (5, 9), (1, 511), (2, 513), (7, 1000), (3, 2047),
                                 (17, 4096), (1, 7168), (300, 2049), (2, 8192), (2, 8193), (2, 16384), (3, 16391),
                                 (1, 32767), (2, 32768)])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_forward_bf16(T, K, kind):
    print("CASE norm", T, K, kind, flush=True)
    check_forward(tokens(T, K, T), None, weight_of(K, kind, 1), 1e-6)
    check_forward(tokens(T, K, T + 1), tokens(T, K, T + 2), weight_of(K, kind, 2), 1e-5, sum_out=T != 5)


@pytest.mark.parametrize("fmt", ["rows", "km", "e8m0"])
@pytest.mark.parametrize("T,K", [(1, 128), (5, 256), (33, 1152), (1, 7168), (130, 2048), (2, 8320), (3, 16512), (1, 32768)])
def test_forward_e4m3(T, K, fmt):
    print("CASE norm e4m3", T, K, fmt, flush=True)
    check_forward(tokens(T, K, T), tokens(T, K, T + 2), weight_of(K, BF16, 1), 1e-6, True, fmt)
    check_forward(tokens(T, K, T + 1), None, weight_of(K, F32, 2), 1e-6, False, fmt)


def test_rows_of_zeros_and_of_very_large_and_small_values():
    K = 1024
    x = tokens(6, K, 3)
    x[1] = 0
    x[2] = (x[2].float() * 2.0 ** 100).to(BF16)              # squares past fp32
    x[3] = (x[3].float() * 2.0 ** -100).to(BF16)             # squares below it: eps alone
    x[4] = torch.finfo(BF16).max
    for fmt in (None, "rows"):
        check_forward(x, None, weight_of(K, F32, 4), 1e-6, True, fmt)
    check_forward(x[:1], None, weight_of(K, F32, 4), 2.0 ** -126)


def test_infinities_and_nan_stay_in_their_rows():
    K = 512
    x = tokens(4, K, 5)
    x[1, 7] = float("inf")
    x[2, 9] = float("nan")
    y, q, qs, rs = buf((4, K), BF16), buf((4, K), E4M3), buf((4, K // 128), F32), buf((4,), F32)
    w = weight_of(K, F32, 6)
    mg.rms_norm(x.cuda(), w.cuda(), y=y, q=q, q_scale=qs, rstd=rs)
    y, q, rs = f64(y), f64(q), f64(rs)
    assert rs[1] == 0 and np.isnan(y[1, 7]) and (np.delete(y[1], 7) == 0).all()
    assert np.isnan(q[1, 7]) and (np.delete(q[1], 7) == 0).all() and (f64(qs)[1] == 1).all()
    assert np.isnan(rs[2]) and np.isnan(y[2]).all() and np.isnan(q[2]).all()
    clean = x[[0, 3]]
    v, _ = ob.rms_norm(clean.double().numpy(), w.double().numpy(), 1e-6)
    assert (np.abs(y[[0, 3]] - v) <= (HALF + 34 * U) * np.abs(v)).all()


def test_sum_in_place():
    x, r, w = tokens(9, 640, 7), tokens(9, 640, 8), weight_of(640, BF16, 9)
    h = (x.float() + r.float()).to(BF16)
    for mine in (0, 1):
        a, b, y = x.cuda(), r.cuda(), buf((9, 640), BF16)
        mg.rms_norm(a, w.cuda(), residual=b, sum_out=(a, b)[mine], y=y)
        assert torch.equal((a, b)[mine].cpu(), h) and torch.equal((b, a)[mine].cpu(), (r, x)[mine])
        v, _ = ob.rms_norm(h.double().numpy(), w.double().numpy(), 1e-6)
        assert (np.abs(f64(y) - v) <= (HALF + 34 * U) * np.abs(v)).all()


def test_bf16_at_any_even_address():
    T, K = 4, 777
    hold = torch.zeros(T * K + 1, dtype=BF16)
    hold[1:] = tokens(T, K, 11).reshape(-1)
    x = hold.cuda()[1:].view(T, K)
    w = torch.cat([torch.zeros(1), weight_of(K, F32, 12)]).cuda()[1:]
    out = buf((1, T * K + 1), BF16)[0]
    mg.rms_norm(x, w, y=out[1:].view(T, K))
    v, _ = ob.rms_norm(f64(x), f64(w), 1e-6)
    assert (np.abs(f64(out[1:].view(T, K)) - v) <= (HALF + 34 * U) * np.abs(v)).all()
    assert out[:1].view(torch.uint8).eq(SENTINEL).all()


# ------------------------------------------------------------------ backward

def check_backward(dy, h, w, rstd, ds=None, want_weight=True):
    T, K = dy.shape
    dx, dw = buf((T, K), BF16), buf((K,), F32) if want_weight else None
    mg.rms_norm_backward(dy.cuda(), h.cuda(), w.cuda(), rstd.cuda(), dx, dw,
                         mg.rms_norm_workspace(T, K) if want_weight else None, d_sum=None if ds is None else ds.cuda())
    torch.cuda.synchronize()
    D, H, W, R = (v.double().numpy() for v in (dy, h, w, rstd))
    S = 0.0 if ds is None else ds.double().numpy()
    rx, rw = ob.rms_norm_backward(D, H, W, R, None if ds is None else S)
    g, xhat = D * W, H * R[:, None]
    M, mean = np.abs(g * xhat).mean(1, keepdims=True), np.abs((g * xhat).mean(1, keepdims=True))
    err = R[:, None] * (3 * U * np.abs(g) + np.abs(xhat) * (58 * U * M + 4 * U * mean)) + U * (np.abs(rx) + np.abs(S))
    assert (np.abs(f64(dx) - rx) <= err + HALF * (np.abs(rx) + err) + 2.0 ** -133).all()
    if want_weight:
        lim = ((T + 255) // 256 + 34) * U * np.abs(D * xhat).sum(0) + 2.0 ** -126
        assert (np.abs(f64(dw) - rw) <= lim).all()
    return dx, dw


def backward_case(T, K, kind, seed):
    g = gen(seed)
    h, w = tokens(T, K, seed), weight_of(K, kind, seed + 1)
    dy, ds = torch.randn(T, K, generator=g).to(BF16), torch.randn(T, K, generator=g).to(BF16)
    rstd = torch.from_numpy(ob.rms_norm(h.double().numpy(), w.double().numpy(), 1e-6)[1]).float()
    return dy, h, w, rstd, ds


@pytest.mark.parametrize("T,K", [(1, 1), (1, 3), (2, 8), (3, 513), (255, 64), (256, 65), (257, 100), (600, 1000), (5, 7168),
                                 (1, 8192), (2, 8193), (3, 16384), (300, 16385), (2, 32768)])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_backward(T, K, kind):
    print("CASE norm backward", T, K, kind, flush=True)
    dy, h, w, rstd, ds = backward_case(T, K, kind, T + K)
    check_backward(dy, h, w, rstd, ds)
    check_backward(dy, h, w, rstd)
    check_backward(dy, h, w, rstd, ds, want_weight=False)


def test_backward_of_rows_of_very_large_values_and_zeros():
    dy, h, w, rstd, ds = backward_case(5, 512, F32, 3)
    h[1] = (h[1].float() * 2.0 ** 100).to(BF16)
    h[2] = 0
    rstd = torch.from_numpy(ob.rms_norm(h.double().numpy(), w.double().numpy(), 1e-6)[1]).float()
    check_backward(dy, h, w, rstd, ds)


def test_backward_in_place():
    dy, h, w, rstd, ds = backward_case(270, 321, BF16, 4)
    want, dw = check_backward(dy, h, w, rstd, ds)
    ws = mg.rms_norm_workspace(270, 321)
    for i in range(3):
        ts = [v.cuda() for v in (dy, h, ds)]
        got = buf((321,), F32)
        mg.rms_norm_backward(ts[0], ts[1], w.cuda(), rstd.cuda(), ts[i], got, ws, d_sum=ts[2])
        assert torch.equal(ts[i], want) and torch.equal(got, dw)


def test_no_tokens():
    w = weight_of(256, F32, 1).cuda()
    e = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    mg.rms_norm(e(0, 256), w, y=e(0, 256), q=e(0, 256, dtype=E4M3), q_scale=e(0, 2, dtype=F32))
    dw = buf((256,), F32)
    mg.rms_norm_backward(e(0, 256), e(0, 256), w, e(0, dtype=F32), e(0, 256), dw, mg.rms_norm_workspace(0, 256))
    assert (f64(dw) == 0).all()


def test_gradients_by_differences():
    """dx against differences of what the calls return: f = sum_k dy h rstd w as a function of one h, with rstd from the
    call.  With r = rstd and g = dy w the third derivative is at most 30 |g| r^3 / K (that of r 24 r^4 / K^1.5, its second
    2 r^3 / K, |h| <= K^.5 / r), r taken 10 % larger for the interval; rstd is off by 32 u, |f| <= |g| |h| r."""
    T, K, eps, step = 2, 16, 0.05, 0.125
    g = gen(9)
    x, w = torch.randint(-8, 9, (T, K), generator=g).to(BF16), torch.randint(1, 5, (K,), generator=g).float()
    dy = torch.randint(-4, 5, (T, K), generator=g).to(BF16)

    def rstd_of(v):
        rs = buf((T,), F32)
        mg.rms_norm(v.cuda(), w.cuda(), y=buf((T, K), BF16), rstd=rs, eps=eps)
        return rs
    rs, dx = rstd_of(x), buf((T, K), BF16)
    mg.rms_norm_backward(dy.cuda(), x.cuda(), w.cuda(), rs, dx)
    for t, c in [(0, 0), (0, 7), (1, 15)]:
        f = []
        for sign in (1, -1):
            v = x.clone()
            v[t, c] += sign * step                           # eighths of whole numbers up to 9: exact in bf16
            f.append(float((dy.double() * v.double() * rstd_of(v).cpu().double()[:, None] * w.double())[t].sum()))
        slope = (f[0] - f[1]) / (2 * step)
        r, G = 1.1 * float(rs[t]), float((dy[t].double() * w.double()).norm())
        lim = 30 / K * r ** 3 * G * step ** 2 / 6 + 32 * U * G * (float(x[t].double().norm()) + step) * r / step
        lim += HALF * (abs(slope) + lim) + 64 * U * G * r
        assert abs(float(dx[t, c]) - slope) <= lim, (t, c, float(dx[t, c]), slope, lim)


def test_graph_and_stream():
    T, K = 37, 1024
    x, r, so, y, dx, dy = (torch.empty(T, K, dtype=BF16, device="cuda") for _ in range(6))
    w = weight_of(K, BF16, 1).cuda()
    q, qs = torch.empty(T, K, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(K // 128, T, device="cuda")
    rs, dw, ws = torch.empty(T, device="cuda"), torch.empty(K, device="cuda"), mg.rms_norm_workspace(T, K)

    def step():
        mg.rms_norm(x, w, residual=r, sum_out=so, y=y, q=q, q_scale=qs, rstd=rs, scale_km=True)
        mg.rms_norm_backward(dy, so, w, rs, dx, dw, ws, d_sum=y)

    def fill(seed):
        for i, v in enumerate((x, r, dy)):
            v.copy_(tokens(T, K, seed + i))
    outs = (so, y, q.view(torch.uint8), qs, rs, dx, dw)
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
