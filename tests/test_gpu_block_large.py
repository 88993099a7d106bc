"""Offsets past 2^32 bytes in the operators around the layer: the last rows against the fp64 oracle (oracle/block.py), with
the bounds of test_gpu_norm.py, test_gpu_balance.py and test_gpu_lora.py."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from oracle import block as ob
from tests.test_gpu_layer import U, f64, gen

pytestmark = pytest.mark.gpu
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def with_last(shape, last, dtype):
    """Zeros on the device, with `last` in the last rows."""
    t = torch.zeros(shape, dtype=dtype, device="cuda")
    t[-len(last):] = last.cuda()
    return t


def test_norm_both_ways():
    T, K, n = 70001, 32768, 3
    assert T * K * 2 > 1 << 32
    g = gen(1)
    h, dy, w = (torch.randn(n, K, generator=g).to(BF16), torch.randn(n, K, generator=g).to(BF16),
                1 + 0.2 * torch.randn(K, generator=g))
    x, y, rstd = with_last((T, K), h, BF16), torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(T, device="cuda")
    mg.rms_norm(x, w.cuda(), y=y, rstd=rstd)
    v, r = ob.rms_norm(h.double().numpy(), w.double().numpy(), 1e-6)
    assert (np.abs(f64(rstd[-n:]) - r) <= 32 * U * r).all() and not bool(y[:-n].any())
    assert (np.abs(f64(y[-n:]) - v) <= (HALF + 34 * U) * np.abs(v) + 2.0 ** -133).all()
    d, dw = with_last((T, K), dy, BF16), torch.empty(K, device="cuda")
    mg.rms_norm_backward(d, x, w.cuda(), rstd, y, dw, mg.rms_norm_workspace(T, K))
    D, H, W, R = dy.double().numpy(), h.double().numpy(), w.double().numpy(), f64(rstd[-n:])
    rx, rw = ob.rms_norm_backward(D, H, W, R)
    gw, xhat = D * W, H * R[:, None]
    M, mean = np.abs(gw * xhat).mean(1, keepdims=True), np.abs((gw * xhat).mean(1, keepdims=True))
    err = R[:, None] * (3 * U * np.abs(gw) + np.abs(xhat) * (58 * U * M + 4 * U * mean)) + U * np.abs(rx)
    assert (np.abs(f64(y[-n:]) - rx) <= err + HALF * (np.abs(rx) + err) + 2.0 ** -133).all()
    # the other rows add exact zeros: the last ones' chain alone
    assert (np.abs(f64(dw) - rw) <= 38 * U * np.abs(D * xhat).sum(0) + 2.0 ** -126).all()


def test_balance_both_ways():
    T, E, k, n = 1100003, 1024, 2, 5
    assert T * E * 4 > 1 << 32
    g = gen(2)
    last, ids = torch.randn(n, E, generator=g), torch.randint(0, E, (n, k), generator=g).to(I32)
    logits, all_ids = with_last((T, E), last, F32), with_last((T, k), ids, I32)
    off = torch.tensor([0, T - n, T], dtype=I32)
    loss, z, probs = torch.empty(2, device="cuda"), torch.empty(2, device="cuda"), torch.empty(2, E, device="cuda")
    counts, d = torch.empty(2, E, dtype=I32, device="cuda"), torch.empty_like(logits)
    mg.balance_loss(logits, all_ids, loss, counts, mg.balance_loss_workspace(T, E, 2), probs=probs, z_loss=z,
                    seq_offsets=off.cuda())
    L = last.double().numpy()
    rl, rz, rc, rp = ob.balance_loss(L, ids.numpy())
    assert int(counts[0, 0]) == (T - n) * k and int(counts[0].sum()) == (T - n) * k
    # p: distances up to 10 of a token's largest logit; five tokens and a few steps of sums
    e = (10 + 26) * 2 * U + 20 * U
    assert np.array_equal(counts[1].cpu().numpy(), rc[0]) and (np.abs(f64(probs[1]) - rp[0]) <= e * rp[0]).all()
    assert abs(float(loss[1]) - rl[0]) <= 2 * e * rl[0] and abs(float(z[1]) - rz[0]) <= 200 * U * rz[0]
    # all logits alike in the first sequence: every p is 1 / E, a power of two, and ln sum e^l is ln E
    assert (np.abs(f64(probs[0]) - 1 / E) <= 8 * U / E + ((T + 255) // 256 + 24) * U / E).all()
    d_loss, d_z = torch.tensor([0.0, 1.0]), torch.tensor([0.0, 0.5])
    mg.balance_loss_backward(logits, counts, d_loss.cuda(), d, k=k, d_z_loss=d_z.cuda(), seq_offsets=off.cuda())
    ref = ob.balance_loss_backward(L, rc, np.array([1.0]), k, np.array([0.5]))
    p = ob.probabilities(L, "softmax")
    c = E / (k * n * n) * rc[0] + (p * E / (k * n * n) * rc[0]).sum(1, keepdims=True)
    lim = p * (c + np.abs(ob.log_sum_exp(L))[:, None] / n) * 200 * U
    assert not bool(d[:-n].any()) and (np.abs(f64(d[-n:]) - ref) <= lim).all()


def test_adapters_of_many_rows():
    T, K, N, R, L, n = 280003, 8192, 8, 8, 3, 4
    assert T * K * 2 > 1 << 32
    g = gen(3)
    x, A = torch.randn(n, K, generator=g).to(BF16), (torch.randn(L, R, K, generator=g) * K ** -0.5).to(BF16)
    B, Y = torch.randn(L, N, R, generator=g).to(BF16), torch.randn(T, N, generator=g).to(BF16)
    who = torch.randint(-1, L, (T,), generator=g).to(I32)
    who[-n:] = torch.tensor([2, 0, -1, 1])
    X, out = with_last((T, K), x, BF16), torch.empty(T, N, dtype=BF16, device="cuda")
    mg.lora(X, A.cuda(), B.cuda(), who.cuda(), Y.cuda(), out, mg.lora_workspace(T, K, R))
    assert torch.equal(out[:-n].cpu(), Y[:-n])               # rows of zeros add nothing
    a = [v.double().numpy() for v in (x, A, B)]
    ref = ob.lora(*a, who[-n:].numpy(), Y[-n:].double().numpy())
    mag = ob.lora(*[np.abs(v) for v in a], who[-n:].numpy(), np.zeros((n, N)))
    # one part of K: 16 units a wave in one chain, 4 waves; U in two halves
    err = mag * ((16 * 128 + 8) * U + 2.0 ** -16) + 2 * U * np.abs(ref)
    assert (np.abs(f64(out[-n:]) - ref) <= err + HALF * (np.abs(ref) + err)).all()
