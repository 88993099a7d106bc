"""Inner products of the adapters near the end of fp32's range, on MI355X."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_layer import f64
from tests.test_gpu_lora import BF16, F32, I32, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


@pytest.mark.parametrize("T", [1, 70, 300])
def test_inner_products_past_bf16_are_finite(T):
    """U = max of bf16 + 1.5 * 2^119 is a number of fp32 that bf16 rounds to infinity.  Its two halves add up to it, so out is
    U B rounded once; infinities of U stay what they are."""
    K, N, R, top = 8, 16, 8, float(torch.finfo(BF16).max)
    X = torch.zeros(T, K)
    X[:, 0], X[:, 1] = top, 1.5 * 2.0 ** 119
    X[T // 2:, :2] *= -1
    if T > 1:
        X[0, 0], X[1, 0] = float("inf"), -float("inf")
    A = torch.zeros(1, R, K)
    A[0, :, :2] = 1
    B = torch.full((1, N, R), 2.0 ** -103)                   # eight equal terms: every sum is exact
    i = dict(X=X.to(BF16), A=A.to(BF16), B=B.to(BF16), Y=torch.zeros(T, N, dtype=BF16), scale=torch.ones(1, dtype=F32),
             adapter=torch.zeros(T, dtype=I32))
    want = (X.double()[:, :2].sum(1) * 2.0 ** -100).float().to(BF16)
    got = run(i).cpu()
    if T > 1:
        assert torch.equal(got[:2].float(), torch.tensor([[float("inf")], [-float("inf")]]).expand(2, N))
        got, want = got[2:], want[2:]
    assert torch.equal(got, want[:, None].expand(-1, N)), f64(got)[:, 0]
