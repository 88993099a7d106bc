"""RMS norm on MI355X with an eps of the squares' size where these pass fp32.  Bounds as in test_gpu_norm.py."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_norm import BF16, F32, check_forward, weight_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


@pytest.mark.parametrize("T,K", [(1, 1), (3, 2), (5, 64), (6, 1000), (600, 1500), (2, 8192), (2, 20000)])
def test_eps_beside_squares_past_fp32(T, K):
    """Sums of squares, and their mean with eps, up to 2^129 and beyond: eps counts in all of them."""
    print("CASE norm eps", T, K, flush=True)
    x = (1 + 0.9 * torch.rand(T, K, generator=torch.Generator().manual_seed(K))) * 2.0 ** 63
    x = x.to(BF16)
    for row in range(1, T, 2):
        x[row] = (x[row].float() * 2.0 ** -7).to(BF16)               # and rows within fp32 beside them
    for eps in (2.0 ** 127, 2.0 ** 126, 2.0 ** 100, 2.0 ** -20):
        check_forward(x, None, weight_of(K, F32, 1), eps)
