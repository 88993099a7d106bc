"""The last sizes that the operators around the layer take, as their header states them, and the first that they refuse (CPU
only): a call past the checks of its sizes ends at its workspace, and nothing here reaches a launch."""
import re

import pytest

import moe_grouped_gemm_sizes_amd as mg
from tests.test_block_api import BL, LORA, NB
from tests.test_layer_api import UNS, WS, call

HEADER = open(mg.HEADER_PATH).read()


def stated(call_name):
    """The comment in front of a call, in one line."""
    before = HEADER[:HEADER.index(f"moegg_status_t {call_name}(")]
    return re.sub(r"\s*\n \*\s*", " ", before[before.rindex("/*"):])


def test_lora_grid():
    """Chunks of 64 rows times panels of 256 columns."""
    most = int(re.search(r"ceil\(T / 64\) \* ceil\(N / 256\) up to (\d+)", stated("moegg_lora")).group(1))
    last = dict(ws=None, T=64, N=256 * most)                 # one chunk: N past 2^30, refused for that
    assert call("moegg_lora", LORA, last) == UNS
    for chunks in (1 << 18, 100003, 1 << 13, 2 ** 13 - 1):
        panels = most // chunks
        size = dict(ws=None, T=64 * chunks, N=256 * panels)
        assert call("moegg_lora", LORA, size) == WS, size
        assert call("moegg_lora", LORA, dict(size, T=size["T"] - 63, N=size["N"] - 248)) == WS
        assert call("moegg_lora", LORA, dict(size, N=size["N"] + 8)) == UNS, size
    chunks, panels = next((c, most // c) for c in range(2, 1 << 18) if most % c == 0)
    assert call("moegg_lora", LORA, dict(ws=None, T=64 * chunks, N=256 * panels)) == WS
    chunks, panels = next((c, (most + 1) // c) for c in range(2, 1 << 18) if (most + 1) % c == 0)
    assert call("moegg_lora", LORA, dict(ws=None, T=64 * chunks, N=256 * panels)) == UNS


@pytest.mark.parametrize("last,first", [
    (dict(K=1 << 30), dict(K=(1 << 30) + 8)), (dict(N=1 << 30, T=64), dict(N=(1 << 30) + 8, T=64)),
    (dict(T=1 << 24), dict(T=(1 << 24) + 1)), (dict(R=128), dict(R=136))])
def test_lora_sizes(last, first):
    words = stated("moegg_lora")
    assert "K and N up to 2^30" in words and "T up to 2^24" in words and "R = 8..128" in words
    assert call("moegg_lora", LORA, dict(last, ws=None)) == WS
    assert call("moegg_lora", LORA, dict(first, ws=None)) == UNS


def test_norm_sizes():
    words = stated("moegg_rms_norm")
    assert "K = 1..32768" in words and "T up to 2097151" in words
    assert call("moegg_rms_norm_backward", NB, dict(T=2097151, K=32768, ws=None)) == WS
    assert call("moegg_rms_norm_backward", NB, dict(T=2097152, ws=None)) == UNS
    assert call("moegg_rms_norm_backward", NB, dict(K=32769, ws=None)) == UNS


def test_balance_sizes():
    words = stated("moegg_balance_loss")
    assert "T = 0..16773120, E = 1..1024, k = 1..32 (and k <= E), S = 1..65536" in words
    last = dict(T=16773120, E=1024, k=32, S=65536, ws=None)
    assert call("moegg_balance_loss", BL, last) == WS
    for name in ("T", "E", "k", "S"):
        assert call("moegg_balance_loss", BL, dict(last, **{name: last[name] + 1})) == UNS
