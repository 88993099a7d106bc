"""Low-rank adapters on MI355X against the fp64 oracle (oracle/block.py).

Bounds, with u = 2^-24 (half a step of fp32): products of two bf16 are exact in fp32.
- U = X A^T: a wave's part of K is up to ceil(units / (4 splits)) units of 128 columns in one chain of products, then 4
  waves and the splits: c u of the terms' magnitudes.
- U B^T: 2^-16 of U is lost in its two halves; 2 R products in a chain.
- out: scale, Y's addition and two more roundings by u each, then bf16's 2^-8.
"""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from oracle import block as ob
from tests.test_gpu_layer import SENTINEL, U, buf, f64, gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def inputs(T, K, N, R, L, seed):
    g = gen(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)            # noqa: E731
    return dict(X=rnd(T, K).to(BF16), A=(rnd(L, R, K) * K ** -0.5).to(BF16), B=(rnd(L, N, R) * R ** -0.5).to(BF16),
                Y=rnd(T, N).to(BF16), scale=rnd(L), adapter=torch.randint(-1, L + 1, (T,), generator=g).to(I32))


def packed(T, L, seed, longest):
    """Adapters of requests of consecutive rows."""
    g, who = gen(seed), []
    while len(who) < T:
        n = int(torch.randint(1, longest + 1, (1,), generator=g))
        who += [int(torch.randint(-1, L, (1,), generator=g))] * n
    return torch.tensor(who[:T], dtype=I32)


def run(i, scale=True, in_place=False, ws=None, stream=None):
    d = {n: v.cuda() for n, v in i.items()}
    (T, K), R = i["X"].shape, i["A"].shape[1]
    out = d["Y"] if in_place else buf(tuple(i["Y"].shape), BF16)
    mg.lora(d["X"], d["A"], d["B"], d["adapter"], d["Y"], out, mg.lora_workspace(T, K, R) if ws is None else ws,
            scale=d["scale"] if scale else None, stream=stream)
    torch.cuda.synchronize()
    return out


def reference(i, scale=True):
    """(out, bound) in fp64, adapter by adapter."""
    X, A, B, Y = (i[n].double().numpy() for n in "XABY")
    T, K = X.shape
    R, L = A.shape[1], A.shape[0]
    who = i["adapter"].numpy()
    ref, err = Y.copy(), np.zeros_like(Y)
    tiles, units = (T + 1) // 2 if T <= 128 else (T + 63) // 64, (K + 127) // 128
    each = -(-units // (4 * -(-(512 if R <= 32 else 256) // tiles)))
    splits = -(-units // (4 * each))
    chain = (each * 128 + 4 + splits) * U
    for a in range(L):
        rows = np.nonzero(who == a)[0]
        if len(rows) == 0:
            continue
        s = float(i["scale"][a]) if scale else 1.0
        u, mag = X[rows] @ A[a].T, np.abs(X[rows]) @ np.abs(A[a]).T
        add = s * (u @ B[a].T)
        e = abs(s) * ((np.abs(u) * (2.0 ** -16 + (2 * R + 4) * U) + mag * chain) @ np.abs(B[a]).T)
        ref[rows] += add
        err[rows] = e + 2 * U * (np.abs(Y[rows]) + np.abs(add))
    there = (who >= 0) & (who < L)
    err += np.where(there[:, None], 2.0 ** -8 * (np.abs(ref) + err) + 2.0 ** -133, 0.0)
    return ref, err


def check(i, scale=True, **kw):
    got = f64(run(i, scale, **kw))
    ref, err = reference(i, scale)
    d = np.abs(got - ref) - err
    assert (d <= 0).all(), (np.unravel_index(d.argmax(), d.shape), float(d.max()))


@pytest.mark.parametrize("T,K,N,R,L", [
    (1, 8, 8, 8, 1), (1, 64, 72, 8, 3), (2, 40, 256, 16, 2), (15, 512, 264, 24, 4), (16, 520, 1000, 32, 1),
    (17, 1032, 304, 40, 5), (63, 256, 248, 64, 70), (64, 2048, 512, 16, 64), (65, 1000, 520, 72, 2),
    (100, 312, 1024, 128, 9), (130, 7168, 4096, 16, 3), (333, 128, 136, 104, 40), (1, 7168, 4096, 64, 2),
    (700, 640, 776, 48, 11), (40, 16, 32, 128, 1)])
def test_rows_in_any_order(T, K, N, R, L):
    print("CASE lora", T, K, N, R, L, flush=True)
    i = inputs(T, K, N, R, L, T + K)
    check(i)
    check(i, scale=False, in_place=True)


@pytest.mark.parametrize("T,K,N,R,L", [(128, 2048, 64, 8, 9), (129, 2048, 64, 8, 9), (256, 64, 64, 8, 7),
                                       (257, 64, 72, 16, 300), (1000, 128, 264, 32, 1), (4096, 72, 40, 64, 64),
                                       (8192, 40, 8, 8, 1500), (8193, 64, 48, 16, 3), (16500, 32, 24, 128, 9000),
                                       (500, 64, 64, 16, 16383), (500, 64, 64, 16, 16384), (500, 64, 64, 16, 20000)])
def test_many_rows_in_any_order(T, K, N, R, L):
    """Rows sorted by adapter, window by window, or (too many adapters to count) taken as they come."""
    print("CASE lora many", T, K, N, R, L, flush=True)
    i = inputs(T, K, N, R, L, T + L)
    check(i)
    i["adapter"][i["adapter"] % 2 == 0] = -1
    check(i, in_place=True)
    check(i, scale=False)
    i["adapter"][:] = L - 1
    check(i)


@pytest.mark.parametrize("T,K,N,R,L,longest", [(64, 256, 256, 16, 2, 64), (500, 512, 384, 16, 4, 300),
                                               (1000, 320, 512, 64, 9, 40), (4100, 128, 264, 8, 5, 3000),
                                               (257, 1024, 640, 32, 3, 17)])
def test_packed_requests(T, K, N, R, L, longest):
    print("CASE lora packed", T, K, N, R, L, longest, flush=True)
    i = dict(inputs(T, K, N, R, L, T), adapter=packed(T, L, T + 1, longest))
    check(i)


def test_rows_of_one_adapter_in_every_number():
    """1 to 64 rows of a chunk share an adapter, the others have one each."""
    base = inputs(64, 96, 104, 16, 65, 3)
    for n in (1, 2, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64):
        who = torch.arange(64, dtype=I32)
        who[torch.randperm(64, generator=gen(n))[:n]] = 64
        print("CASE lora shared", n, flush=True)
        check(dict(base, adapter=who))


def test_whole_numbers_are_exact():
    """Small integers: every sum is exact, and the result is one rounding of it."""
    g = gen(4)
    whole = lambda *s: torch.randint(-3, 4, s, generator=g).to(BF16)   # noqa: E731
    i = dict(X=whole(90, 264), A=whole(4, 40, 264), B=whole(4, 200, 40), Y=whole(90, 200), scale=torch.full((4,), 0.5),
             adapter=torch.randint(-1, 4, (90,), generator=g).to(I32))
    ref = torch.from_numpy(ob.lora(*(i[n].double().numpy() for n in "XAB"), i["adapter"].numpy(), i["Y"].double().numpy(),
                                   i["scale"].double().numpy()))
    assert torch.equal(run(i).cpu(), ref.float().to(BF16))


def test_rows_without_an_adapter():
    for T in (150, 600):
        _without_an_adapter(inputs(T, 64, 128, 16, 3, 5))


def _without_an_adapter(i):
    i["adapter"][:] = -1
    i["X"][:] = float("nan")                                 # not looked at
    assert torch.equal(run(i).cpu().view(torch.int16), i["Y"].view(torch.int16))
    i["adapter"][::3] = 2 ** 31 - 1
    i["adapter"][1::3] = -2 ** 31
    assert torch.equal(run(i, in_place=True).cpu().view(torch.int16), i["Y"].view(torch.int16))


@pytest.mark.parametrize("T", [130, 390])
def test_nan_and_infinities_stay_in_their_rows_and_adapters(T):
    i = inputs(T, 256, 64, 16, 4, 6)
    i["adapter"] = torch.arange(T, dtype=I32) % 4
    j = {n: v.clone() for n, v in i.items()}
    j["X"][5, 7], j["X"][70, 3] = float("nan"), float("inf")
    j["A"][2, 3] = float("nan")
    j["B"][3, 11] = float("inf")
    a, b = f64(run(i)), f64(run(j))
    hit = np.zeros((T, 64), dtype=bool)
    hit[[5, 70]] = True
    hit[2::4] = True
    hit[3::4, 11] = True
    assert np.array_equal(a[~hit], b[~hit]) and np.isnan(b[5]).all() and np.isnan(b[2::4]).all()
    assert not np.isfinite(b[70]).any() and not np.isfinite(b[3::4, 11]).any()


@pytest.mark.parametrize("T,K,N,R,L", [(77, 72, 88, 24, 5), (300, 72, 88, 24, 5), (8500, 136, 8, 8, 7000)])
def test_nothing_is_written_past_the_outputs(T, K, N, R, L):
    i = inputs(T, K, N, R, L, 7)
    n = mg.lora_workspace_bytes(T, K, R)
    ws = torch.full((n + 512,), SENTINEL, dtype=torch.uint8, device="cuda")
    out = torch.full((2 * T * N + 64,), SENTINEL, dtype=torch.uint8, device="cuda")
    d = {k: v.cuda() for k, v in i.items()}
    mg.lora(d["X"], d["A"], d["B"], d["adapter"], d["Y"], out[:-64].view(BF16).view(T, N), ws[:n], scale=d["scale"])
    torch.cuda.synchronize()
    assert bool((ws[n:] == SENTINEL).all()) and bool((out[-64:] == SENTINEL).all())
    assert torch.equal(out[:-64].view(BF16).view(T, N).cpu(), run(i).cpu())


def test_no_rows():
    i = inputs(0, 64, 64, 8, 2, 8)
    run(i)


def test_a_larger_workspace_and_repeated_bits():
    for T in (200, 2000):
        i = inputs(T, 1536, 256, 16, 6, 9)
        a = run(i)
        assert torch.equal(a, run(i, ws=mg.lora_workspace(5000, 1536, 16))) and torch.equal(a, run(i))


def test_weights_past_32_bit_offsets():
    """The last adapter of a table of more than 2^32 bytes."""
    K, N, R = 16384, 8, 128
    L = (1 << 32) // (2 * R * K) + 2
    g = gen(10)
    A = torch.zeros(L, R, K, dtype=BF16, device="cuda")
    i = dict(X=torch.randn(3, K, generator=g).to(BF16), A=(torch.randn(1, R, K, generator=g) * K ** -0.5).to(BF16),
             B=torch.randn(1, N, R, generator=g).to(BF16), Y=torch.randn(3, N, generator=g).to(BF16), scale=torch.ones(1),
             adapter=torch.zeros(3, dtype=I32))
    ref, err = reference(i)
    A[L - 1] = i["A"][0].cuda()
    B = torch.zeros(L, N, R, dtype=BF16, device="cuda")
    B[L - 1] = i["B"][0].cuda()
    out = buf((3, N), BF16)
    mg.lora(i["X"].cuda(), A, B, torch.full((3,), L - 1, dtype=I32, device="cuda"), i["Y"].cuda(), out,
            mg.lora_workspace(3, K, R))
    assert (np.abs(f64(out) - ref) <= err).all()


@pytest.mark.parametrize("T", [140, 1400])
def test_graph_and_stream(T):
    K, N, R, L = 512, 256, 16, 6
    d = {n: v.cuda() for n, v in inputs(T, K, N, R, L, 1).items()}
    out, ws = torch.empty(T, N, dtype=BF16, device="cuda"), mg.lora_workspace(T, K, R)

    def step():
        mg.lora(d["X"], d["A"], d["B"], d["adapter"], d["Y"], out, ws, scale=d["scale"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    first = out.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 20, 30, 1):
        for n, v in inputs(T, K, N, R, L, seed).items():
            d[n].copy_(v)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got, out)
    assert torch.equal(first, out)
