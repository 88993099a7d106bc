"""Token permutation on MI355X at widths past 8192 columns, where combine's backward goes round its columns again:
against the fp64 oracle under the bounds of tests/test_gpu_layer.py.

A weight's gradient: up to 16 waves take 512 columns each, 8 a lane, so a lane sums 8 * ceil(N / 8192) products in a
chain, and 6 + 16 sums of lanes and waves follow: (8 * ceil(N / 8192) + 22) u times the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from oracle import layer as ol
from tests.test_gpu_layer import BF16, U, buf, check_rows_operand, f64, gen, operand, some_rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mg.lib()


@pytest.mark.parametrize("T,k,N,rows,fmt", [
    (5, 9, 8320, 40, "rows"), (5, 9, 8320, 40, "km"), (5, 9, 8320, 40, "e8m0"), (3, 2, 16512, 6, "km"),
    (5, 3, 8193, 14, "bf16"), (4, 9, 12345, 30, "bf16"), (2, 1, 16385, 2, "bf16"), (3, 2, 8192, 6, "rows")])
def test_combine_backward_past_8192_columns(T, k, N, rows, fmt):
    g = gen(N + T)
    dout, Y, w = torch.randn(T, N, generator=g).to(BF16), torch.randn(rows, N, generator=g).to(BF16), torch.rand(T, k, generator=g)
    row_of = some_rows(T, k, rows, 9)
    dY, sc = operand((rows,), rows, N, fmt)
    dw = buf((T, k), torch.float32)
    mg.combine_backward(dout.cuda(), Y.cuda(), w.cuda(), row_of.cuda(), dY, dw, sc, scale_km=fmt == "km")
    rY, rw, mag = ol.combine_backward(f64(dout), f64(Y), f64(w), row_of.numpy(), rows)
    check_rows_operand(dY, sc, rY, fmt, rows)
    assert (np.abs(f64(dw) - rw) <= (8 * -(-N // 8192) + 22) * U * mag).all()


@pytest.mark.parametrize("N", [8193, 16640])
def test_dispatch_and_combine_past_8192_columns(N):
    T, k, rows = 7, 3, 18
    x, w = torch.randn(T, N, generator=gen(N)).to(BF16), torch.rand(T, k, generator=gen(1))
    row_of = some_rows(T, k, rows, 10)
    for fmt in ["bf16"] + (["rows", "km", "e8m0"] if N % 128 == 0 else []):
        A, sc = operand((rows,), rows, N, fmt)
        mg.dispatch(x.cuda(), row_of.cuda(), A, sc, scale_km=fmt == "km")
        check_rows_operand(A, sc, ol.dispatch(f64(x), row_of.numpy(), rows), fmt, rows)
    Y, out = torch.randn(rows, N, generator=gen(2)).to(BF16), buf((T, N), BF16)
    mg.combine(Y.cuda(), row_of.cuda(), out, w.cuda())
    ref, mag = ol.combine(f64(Y), row_of.numpy(), f64(w), rows)
    assert (np.abs(f64(out) - ref) <= 2.0 ** -8 * np.abs(ref) + 1.01 * (k + 1) * U * mag).all()
