"""e4m3 codes and fp32 scales of bf16 values, and of bf16 values times a weight, on MI355X: equal to what
s = amax / 448 (1 where that is 0) and e4m3_rne(x / s) give with both divisions rounded to fp32 (+0 and -0 are equal).

bf16 values over a bf16 maximum lie on e4m3's rounding borders, or within an ulp of them, once in two hundred, so that a
quotient 2 ulp off takes another code there.  The CPU's divisions are correctly rounded."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_layer import BF16, E4M3, gen, operand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def values(rows, width, seed):
    """bf16 values with groups of zeros, of subnormal and tiny scales, and of large ones."""
    x = torch.randn(rows, width, generator=gen(seed))
    x[0, :128] = 0
    x[1, :128] *= 1e-36
    x[2, :128] = 1e-40
    x[3, :128] *= 1e36
    x[4, :128] *= 2.0 ** -101
    return x.to(BF16)


def codes(v, s):
    return (v / s).clamp(-448, 448).to(E4M3).float()


def scale(amax):
    s = amax / 448
    return torch.where(s > 0, s, torch.ones_like(s))


def row_operand(v):
    """fp32 [R, W] -> the codes' values and scales of 1x128 groups."""
    g = v.reshape(v.shape[0], -1, 128)
    s = scale(g.abs().amax(-1))
    return codes(g, s[..., None]).reshape(v.shape), s


def borders(v, s):
    """Values whose quotient is within 2^-22 of a border between two codes (above e4m3's subnormals)."""
    q = v.double() / s.double()
    m = torch.frexp(q)[0].abs() * 16 % 1                    # a border has 4 bits after the leading one, the last set
    return int((((m - 0.5).abs() < 2.0 ** -18) & (q.abs() > 2.0 ** -6)).sum())


@pytest.mark.parametrize("fmt", ["bf16", "rows", "km"])
def test_checkpoint_codes_are_those_of_dispatch(fmt):
    R, I = 300, 640
    gu = values(R, 2 * I, 31)
    want, s = row_operand(gu.float())
    assert borders(gu.float().reshape(R, -1, 128), s[..., None]) > 500
    H, hs = operand((R,), R, I, fmt)
    ck, cs = operand((R,), R, 2 * I, "rows")
    mg.swiglu_checkpoint(gu.cuda(), torch.tensor([R], dtype=torch.int32).cuda(), H, ck, cs, hs, scale_km=fmt == "km")
    assert torch.equal(cs.cpu(), s)
    assert torch.equal(ck.cpu().float(), want)
    A, A_scale = operand((R,), R, 2 * I, "rows")
    mg.dispatch(gu.cuda(), torch.arange(R, dtype=torch.int32).view(R, 1).cuda(), A, A_scale)
    assert torch.equal(A_scale, cs) and torch.equal(A.view(torch.uint8), ck.view(torch.uint8))


@pytest.mark.parametrize("fmt", ["rows", "km", "e8m0"])
def test_combine_backward_codes(fmt):
    """dY = w * dout, rounded to fp32: a common factor leaves the quotients near where they were."""
    T, k, N = 60, 3, 1152
    dout = values(T, N, 32)
    w = torch.rand(T, k, generator=gen(33))
    w[7] = torch.tensor([1.0, 0.0, 0.5])
    w[8] = torch.tensor([-0.7, 2.0 ** -20, 3.0])
    v = (w[:, :, None] * dout.float()[:, None, :]).reshape(T * k, N)
    Y = torch.randn(T * k, N, generator=gen(34)).to(BF16)
    dY, sc = operand((T * k,), T * k, N, fmt)
    dw = torch.empty(T, k, device="cuda")
    mg.combine_backward(dout.cuda(), Y.cuda(), w.cuda(), torch.arange(T * k, dtype=torch.int32).view(T, k).cuda(), dY, dw,
                        sc, scale_km=fmt == "km")
    want, s = row_operand(v)
    if fmt == "e8m0":                                       # the power of two that is at least s
        m, e = torch.frexp(s)
        e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
        assert torch.equal(sc.t().cpu().int(), e + 127)
        want = codes(v.reshape(T * k, -1, 128), torch.ldexp(torch.ones_like(s), e)[..., None]).reshape(v.shape)
    else:
        assert torch.equal((sc.t() if fmt == "km" else sc).cpu(), s)
    assert torch.equal(dY.cpu().float(), want)


def test_token_group_codes_of_bf16_rows():
    counts, M = [300, 0, 128, 5, 77], 512
    R = sum(counts)
    x = torch.randn(R, M, generator=gen(35))
    x[:, 7] = 0
    x[:, 300] *= 1e-36
    x[:, 301] *= 1e-38
    x[:, 302] *= 1e36
    x = x.to(BF16)
    S = mg.k_scale_groups(counts)
    X_k, ks = torch.empty(R, M, dtype=torch.uint8, device="cuda").view(E4M3), torch.empty(S, M, device="cuda")
    mg.checkpoint_to_k_groups(x.cuda(), torch.tensor(counts, dtype=torch.int32).cuda(), X_k, ks)
    at = n = near = 0
    for c in counts:
        for r in range(at, at + c, 128):
            v = x[r:min(r + 128, at + c)].float()
            s = scale(v.abs().amax(0))
            near += borders(v, s)
            assert torch.equal(ks[n].cpu(), s)
            assert torch.equal(X_k.cpu()[r:r + v.shape[0]].float(), codes(v, s))
            n += 1
        at += c
    assert n == S and near > 500
