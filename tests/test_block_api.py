"""Refusals of the operators around the layer (CPU only): the C ABI's host checks, and the binding's checks of every
tensor it hands over.  Nothing here reaches a launch."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg
from tests.test_layer_api import EIGHT, FAKE, INV, ODD, UNS, WS, call

E4M3, BF16, F32, I32, U8 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32, torch.uint8
TWO = ctypes.c_void_p(0x100002)
NAN, INF = float("nan"), float("inf")

NORM = dict(x=FAKE, residual=FAKE, weight=FAKE, kind=mg.WEIGHT_BF16, eps=1e-6, sum_out=FAKE, y=FAKE, q=FAKE, q_scale=FAKE,
            rstd=FAKE, T=100, K=256, dtype=mg.FP8_E4M3)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), INV), (dict(weight=None), INV), (dict(q=None), INV), (dict(q_scale=None), INV),
    (dict(residual=None), INV),                              # a sum without a residual
    (dict(dtype=mg.BF16), INV), (dict(dtype=mg.BF16, q=None, q_scale=None, y=None), INV),
    (dict(dtype=mg.BF16, q_scale=None), INV), (dict(dtype=mg.FP8_E4M3_FP4_E2M1), INV), (dict(dtype=17), INV),
    (dict(kind=2), INV), (dict(kind=-1), INV), (dict(T=-1), INV), (dict(K=0), INV), (dict(K=-128), INV),
    (dict(eps=0.0), INV), (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV), (dict(eps=1e-40), INV),
    (dict(x=EIGHT), INV), (dict(residual=EIGHT), INV), (dict(sum_out=EIGHT), INV), (dict(y=EIGHT), INV),
    (dict(q=EIGHT), INV), (dict(weight=EIGHT), INV), (dict(q_scale=TWO), INV), (dict(rstd=TWO), INV),
    (dict(dtype=mg.BF16, q=None, q_scale=None, x=ODD), INV),
    (dict(dtype=mg.BF16, q=None, q_scale=None, weight=TWO, kind=mg.WEIGHT_FP32), INV),
    (dict(K=200), UNS), (dict(K=32896), UNS), (dict(T=1 << 21), UNS),
    (dict(dtype=mg.BF16, q=None, q_scale=None, K=32769), UNS),
])
def test_rms_norm_refusals(kw, status):
    assert call("moegg_rms_norm", NORM, kw) == status


NB = dict(dy=FAKE, h=FAKE, weight=FAKE, kind=mg.WEIGHT_BF16, rstd=FAKE, d_sum=FAKE, dx=FAKE, d_weight=FAKE, T=100, K=250,
          ws=FAKE, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), INV), (dict(h=None), INV), (dict(weight=None), INV), (dict(rstd=None), INV), (dict(dx=None), INV),
    (dict(kind=3), INV), (dict(T=-1), INV), (dict(K=0), INV), (dict(dy=ODD), INV), (dict(h=ODD), INV),
    (dict(d_sum=ODD), INV), (dict(dx=ODD), INV), (dict(rstd=TWO), INV), (dict(d_weight=TWO), INV),
    (dict(weight=TWO, kind=mg.WEIGHT_FP32), INV), (dict(K=32769), UNS), (dict(T=1 << 21), UNS),
    (dict(ws=None), WS), (dict(ws=EIGHT), WS), (dict(ws_bytes=1000), WS),
])
def test_rms_norm_backward_refusals(kw, status):
    assert call("moegg_rms_norm_backward", NB, kw) == status


BL = dict(logits=FAKE, kind=mg.LOGITS_FP32, ids=FAKE, offsets=FAKE, loss=FAKE, z_loss=FAKE, counts=FAKE, probs=FAKE, T=100,
          E=64, k=8, S=3, score=mg.SCORE_SOFTMAX, ws=FAKE, ws_bytes=1 << 20)
BALANCE_BAD = [
    (dict(logits=None), INV), (dict(counts=None), INV), (dict(offsets=None), INV), (dict(T=-1), INV), (dict(E=0), INV),
    (dict(k=0), INV), (dict(k=65), INV), (dict(S=0), INV), (dict(kind=2), INV), (dict(score=2), INV),
    (dict(logits=TWO), INV), (dict(kind=mg.LOGITS_BF16, logits=ODD), INV), (dict(offsets=TWO), INV),
    (dict(counts=TWO), INV), (dict(T=16773121), UNS), (dict(E=1025), UNS), (dict(k=33), UNS), (dict(S=65537), UNS),
    (dict(score=mg.SCORE_SIGMOID), UNS),                     # no z loss of sigmoids
]


@pytest.mark.parametrize("kw,status", BALANCE_BAD + [
    (dict(ids=None), INV), (dict(loss=None), INV), (dict(ids=TWO), INV), (dict(loss=TWO), INV), (dict(z_loss=TWO), INV),
    (dict(probs=TWO), INV), (dict(ws=None), WS), (dict(ws=EIGHT), WS), (dict(ws_bytes=100), WS),
])
def test_balance_loss_refusals(kw, status):
    assert call("moegg_balance_loss", BL, kw) == status


BB = dict(logits=FAKE, kind=mg.LOGITS_FP32, counts=FAKE, offsets=FAKE, d_loss=FAKE, d_z=FAKE, before=FAKE, d_logits=FAKE,
          T=100, E=64, k=8, S=3, score=mg.SCORE_SOFTMAX)


@pytest.mark.parametrize("kw,status", BALANCE_BAD + [
    (dict(d_loss=None), INV), (dict(d_logits=None), INV), (dict(d_loss=TWO), INV), (dict(d_z=TWO), INV),
    (dict(before=TWO), INV), (dict(d_logits=TWO), INV),
])
def test_balance_loss_backward_refusals(kw, status):
    assert call("moegg_balance_loss_backward", BB, kw) == status


LORA = dict(X=FAKE, A=FAKE, B=FAKE, scale=FAKE, adapter=FAKE, Y=FAKE, out=FAKE, T=100, K=256, N=512, R=16, L=4, ws=FAKE,
            ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), INV) for n in ("X", "A", "B", "adapter", "Y", "out")] + [
    (dict([(n, EIGHT)]), INV) for n in ("X", "A", "B", "Y", "out")] + [
    (dict(scale=TWO), INV), (dict(adapter=TWO), INV), (dict(T=-1), INV), (dict(K=0), INV), (dict(N=0), INV),
    (dict(R=0), INV), (dict(L=0), INV), (dict(K=-8), INV), (dict(K=260), UNS), (dict(N=4), UNS), (dict(R=12), UNS),
    (dict(R=136), UNS), (dict(T=(1 << 24) + 1), UNS), (dict(T=1 << 24, N=1 << 20), UNS), (dict(K=(1 << 30) + 8), UNS),
    (dict(N=(1 << 30) + 8), UNS), (dict(ws=None), WS), (dict(ws=EIGHT), WS), (dict(ws_bytes=100), WS),
])
def test_lora_refusals(kw, status):
    assert call("moegg_lora", LORA, kw) == status


def test_workspace_bytes():
    L = mg.lib()
    n, b, a = L.moegg_rms_norm_workspace_bytes, L.moegg_balance_loss_workspace_bytes, L.moegg_lora_workspace_bytes
    assert n(-1, 8) == n(8, 0) == n(8, 32769) == b(-1, 8, 1) == b(8, 0, 1) == b(8, 8, 0) == b(8, 1025, 1) == 0
    assert a(-1, 8, 8) == a(8, 9, 8) == a(8, 8, 4) == a(8, 8, 136) == a((1 << 24) + 1, 8, 8) == 0
    for f in (lambda t: n(t, 7168), lambda t: b(t, 256, 16), lambda t: a(t, 7168, 16)):
        sizes = [f(t) for t in [*range(3000), 8191, 8192, 8193, 32768, 32769, 100000, 1 << 20]]
        assert sizes == sorted(sizes) and sizes[0] > 0       # of T tokens: serves every smaller call
        assert all(s % 256 == 0 for s in sizes)
    assert [b(5000, 64, s) for s in range(1, 300)] == sorted(b(5000, 64, s) for s in range(1, 300))


# ------------------------------------------------------------------ the binding

def t(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=torch.uint8).view(dtype) if dtype is E4M3 else torch.zeros(shape, dtype=dtype)


def bad(match, f, *a, **kw):
    with pytest.raises(ValueError, match=match):
        f(*a, **kw)


def test_rms_norm_binding():
    x, w = t(4, 256), t(256)
    bad("x", mg.rms_norm, t(4, 256, dtype=F32), w, y=t(4, 256))
    bad("y or q", mg.rms_norm, x, w)
    bad("weight", mg.rms_norm, x, t(255), y=t(4, 256))
    bad("weight", mg.rms_norm, x, t(256, dtype=torch.float16), y=t(4, 256))
    bad("weight", mg.rms_norm, x, None, y=t(4, 256))
    bad("y", mg.rms_norm, x, w, y=t(4, 255))
    bad("sum_out", mg.rms_norm, x, w, y=t(4, 256), sum_out=t(4, 256))
    bad("residual", mg.rms_norm, x, w, y=t(4, 256), residual=t(3, 256))
    bad("q_scale", mg.rms_norm, x, w, y=t(4, 256), q_scale=t(4, 2, dtype=F32))
    bad("scale_km", mg.rms_norm, x, w, y=t(4, 256), scale_km=True)
    bad("q", mg.rms_norm, x, w, q=t(4, 256), q_scale=t(4, 2, dtype=F32))
    bad("q", mg.rms_norm, x, w, q=t(3, 256, dtype=E4M3), q_scale=t(3, 2, dtype=F32))
    bad("q_scale", mg.rms_norm, x, w, q=t(4, 256, dtype=E4M3), q_scale=t(2, 4, dtype=F32))
    bad("q_scale", mg.rms_norm, x, w, q=t(4, 256, dtype=E4M3))
    bad("multiple of 128", mg.rms_norm, t(4, 200), t(200), q=t(4, 200, dtype=E4M3), q_scale=t(4, 1, dtype=F32))
    bad("rstd", mg.rms_norm, x, w, y=t(4, 256), rstd=t(5, dtype=F32))
    bad("device tensor", mg.rms_norm, x, w, y=t(4, 256))


def test_rms_norm_backward_binding():
    a = dict(dy=t(4, 64), h=t(4, 64), weight=t(64), rstd=t(4, dtype=F32), dx=t(4, 64), d_weight=t(64, dtype=F32),
             ws=t(1 << 16, dtype=U8))
    f = lambda **kw: mg.rms_norm_backward(**dict(a, **kw))   # noqa: E731
    for name, v in [("h", t(4, 65)), ("rstd", t(4)), ("dx", t(3, 64)), ("d_weight", t(64)), ("weight", t(65)),
                    ("d_sum", t(4, 63)), ("ws", t(16, dtype=U8)), ("ws", None), ("dy", t(4, 64, dtype=F32))]:
        bad(name, f, **{name: v})
    bad("device tensor", f)


def test_balance_binding():
    a = dict(logits=t(6, 8, dtype=F32), ids=t(6, 2, dtype=I32), loss=t(1, dtype=F32), counts=t(1, 8, dtype=I32),
             ws=t(1 << 16, dtype=U8))
    f = lambda **kw: mg.balance_loss(**dict(a, **kw))        # noqa: E731
    for name, v in [("ids", t(5, 2, dtype=I32)), ("loss", t(2, dtype=F32)), ("counts", t(1, 7, dtype=I32)),
                    ("probs", t(1, 7, dtype=F32)), ("z_loss", t(3, dtype=F32)), ("seq_offsets", t(3, dtype=I32)),
                    ("ws", t(16, dtype=U8)), ("ws", None), ("logits", t(6, 8, dtype=torch.float16))]:
        bad(name, f, **{name: v})
    bad("seq_offsets", f, counts=t(2, 8, dtype=I32), loss=t(2, dtype=F32))
    bad("device tensor", f)
    b = dict(logits=t(6, 8), counts=t(1, 8, dtype=I32), d_loss=t(1, dtype=F32), d_logits=t(6, 8), k=2)
    f = lambda **kw: mg.balance_loss_backward(**dict(b, **kw))   # noqa: E731
    for name, v in [("d_logits", t(6, 8, dtype=F32)), ("before", t(6, 8, dtype=F32)), ("d_loss", t(2, dtype=F32)),
                    ("d_z_loss", t(1)), ("counts", t(1, 9, dtype=I32))]:
        bad(name, f, **{name: v})
    bad("seq_offsets", f, counts=t(2, 8, dtype=I32), d_loss=t(2, dtype=F32))
    bad("device tensor", f)


def test_lora_binding():
    a = dict(X=t(5, 64), A=t(3, 8, 64), B=t(3, 32, 8), adapter=t(5, dtype=I32), Y=t(5, 32), out=t(5, 32),
             ws=t(1 << 16, dtype=U8))
    f = lambda **kw: mg.lora(**dict(a, **kw))                # noqa: E731
    for name, v in [("X", t(5, 64, dtype=F32)), ("A", t(3, 8, 63)), ("A", t(8, 64)), ("A", None), ("B", t(2, 32, 8)),
                    ("B", t(3, 8, 32)), ("adapter", t(5, dtype=torch.int64)), ("adapter", t(4, dtype=I32)),
                    ("out", t(5, 31)), ("scale", t(4, dtype=F32)), ("ws", t(16, dtype=U8)), ("ws", None)]:
        bad(name, f, **{name: v})
    bad("device tensor", f)
