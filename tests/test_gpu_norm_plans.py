"""RMS norm on MI355X where its launch takes other plans than for few or narrow rows (more than 512 of them, wide or of odd
width: 16 columns a thread, and several rows of several waves a workgroup), and its backward pass in place past 8192 columns.
Bounds as in test_gpu_norm.py."""
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_gpu_layer import buf
from tests.test_gpu_norm import BF16, F32, backward_case, check_backward, check_forward, tokens, weight_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


@pytest.mark.parametrize("T,K", [(513, 4097), (513, 4104), (520, 7168), (514, 8192), (513, 8191), (600, 1025), (601, 2047),
                                 (1025, 1500), (700, 2051), (513, 1024), (2049, 72)])
@pytest.mark.parametrize("kind", [BF16, F32])
def test_more_than_512_rows(T, K, kind):
    print("CASE norm rows", T, K, kind, flush=True)
    x = tokens(T, K, T)
    x[1], x[T - 1] = 0, (x[T - 1].float() * 2.0 ** 100).to(BF16)     # of zeros, and squares past fp32
    check_forward(x, tokens(T, K, T + 1), weight_of(K, kind, 1), 1e-6)
    check_forward(x, None, weight_of(K, kind, 2), 1e-5)


@pytest.mark.parametrize("fmt", ["rows", "km", "e8m0"])
@pytest.mark.parametrize("T,K", [(513, 4224), (600, 7168), (777, 256)])
def test_more_than_512_rows_e4m3(T, K, fmt):
    print("CASE norm rows e4m3", T, K, fmt, flush=True)
    check_forward(tokens(T, K, T), tokens(T, K, T + 1), weight_of(K, BF16, 1), 1e-6, True, fmt)


@pytest.mark.parametrize("T,K", [(70, 8200), (40, 16384), (30, 16395), (20, 32768)])
def test_backward_in_place_of_wide_rows(T, K):
    print("CASE norm in place", T, K, flush=True)
    dy, h, w, rstd, ds = backward_case(T, K, BF16, 4)
    want, dw = check_backward(dy, h, w, rstd, ds)
    ws = mg.rms_norm_workspace(T, K)
    for i in range(3):
        ts = [v.cuda() for v in (dy, h, ds)]
        got = buf((K,), F32)
        mg.rms_norm_backward(ts[0], ts[1], w.cuda(), rstd.cuda(), ts[i], got, ws, d_sum=ts[2])
        assert torch.equal(ts[i], want) and torch.equal(got, dw)
