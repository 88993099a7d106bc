"""Widths that the layer calls cannot index are refused (CPU only): nothing here reaches a launch."""
import pytest

import moe_grouped_gemm_sizes_amd as mg
from tests.test_layer_api import CB, COMBINE, DISPATCH, call


@pytest.mark.parametrize("width", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 31 - 8191, 2 ** 30 + 128])
@pytest.mark.parametrize("T", [0, 1, 8])
@pytest.mark.parametrize("dtype", [mg.BF16, mg.FP8_E4M3])
def test_widths_past_32_bit_columns(width, T, dtype):
    """Columns are counted in 32 bits, in steps of up to 8192."""
    assert call("moegg_dispatch", DISPATCH, dict(T=T, k=1, K=width, dtype=dtype)) == mg.ERR_UNSUPPORTED
    assert call("moegg_combine", COMBINE, dict(T=T, k=1, N=width)) == mg.ERR_UNSUPPORTED
    assert call("moegg_combine_backward", CB, dict(T=T, k=1, N=width, dtype=dtype)) == mg.ERR_UNSUPPORTED
