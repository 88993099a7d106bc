"""e4m3 codes and scales of the norm on MI355X: equal to what s = amax / 448 (1 where that is 0; E8M0: the power of two that
is at least it) and e4m3_rne(v / s) give for v = h rstd weight with every product and division rounded to fp32 and the rstd
that the call wrote (+0 and -0 are equal).

v is a bf16 value times a factor that its row shares, so that quotients lie on e4m3's rounding borders, or within an ulp of
them, far more often than by chance, and a quotient 2 ulp off takes another code there."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_layer import BF16, E4M3, gen, operand
from tests.test_gpu_layer_codes import borders, codes, row_operand

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


def weights(K, kind):
    """Groups of zeros, of tiny and of large weights, of equal ones and of any."""
    w = 1 + 0.1 * torch.randn(K, generator=gen(2))
    w[:128] = 0
    w[128:256] *= 1e-36
    w[256:384] *= 1e36
    w[384:512] *= 2.0 ** -101
    w[512:1024] = 1
    return w.to(kind)


@pytest.mark.parametrize("fmt", ["rows", "km", "e8m0"])
@pytest.mark.parametrize("T,K,kind", [(300, 1280, BF16), (40, 7168, F32), (9, 16640, BF16), (600, 4224, F32)])
def test_codes_are_those_of_the_rounded_quotient(T, K, kind, fmt):
    print("CASE norm codes", T, K, kind, fmt, flush=True)
    x, r = torch.randn(T, K, generator=gen(T)).to(BF16), torch.randn(T, K, generator=gen(T + 1)).to(BF16)
    w = weights(K, kind)
    q, qs = operand((T,), T, K, fmt)
    y, rstd = torch.empty(T, K, dtype=BF16, device="cuda"), torch.empty(T, device="cuda")
    mg.rms_norm(x.cuda(), w.cuda(), residual=r.cuda(), y=y, q=q, q_scale=qs, rstd=rstd, scale_km=fmt == "km")
    h = (x.float() + r.float()).to(BF16).float()
    v = h * rstd.cpu()[:, None] * w.float()
    assert torch.equal(y.cpu(), v.to(BF16))
    want, s = row_operand(v)
    if fmt == "e8m0":
        m, e = torch.frexp(s)
        e = torch.where(m == 0.5, e - 1, e).clamp(min=-126)
        assert torch.equal(qs.t().cpu().int(), e + 127)
        want = codes(v.reshape(T, -1, 128), torch.ldexp(torch.ones_like(s), e)[..., None]).reshape(v.shape)
    else:
        # one value in two hundred of the four groups of equal weights: 2.5 a row, and those of other weights beside them
        assert borders(v.reshape(T, -1, 128), s[..., None]) > 2 * T
        assert torch.equal((qs.t() if fmt == "km" else qs).cpu(), s)
    assert torch.equal(q.cpu().float(), want), int((q.cpu().float() != want).sum())
