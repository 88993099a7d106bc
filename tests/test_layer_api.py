"""Refusals of the layer operators (CPU only): the C ABI's host checks, and the binding's checks of every tensor it
hands over.  Nothing here reaches a launch."""
import ctypes

import pytest
import torch

import moe_grouped_gemm_sizes_amd as mg

E4M3, BF16, F32, I32, U8 = torch.float8_e4m3fn, torch.bfloat16, torch.float32, torch.int32, torch.uint8
FAKE = ctypes.c_void_p(0x100000)        # aligned, never dereferenced: validation fails first
ODD, EIGHT = ctypes.c_void_p(0x100001), ctypes.c_void_p(0x100008)
INV, UNS, WS = mg.ERR_INVALID_ARG, mg.ERR_UNSUPPORTED, mg.ERR_WORKSPACE


def call(name, defaults, kw):
    args = dict(defaults)
    for k in kw:
        assert k in args, k
    args.update(kw)
    return getattr(mg.lib(), name)(*args.values(), None)


ROUTE = dict(logits=FAKE, kind=mg.LOGITS_FP32, bias=None, ids=FAKE, weights=FAKE, m_sizes=FAKE, row_of=FAKE, T=100, E=64,
             k=8, score=0, n_groups=1, topk_groups=1, group_top=1, renorm=1, scale=1.0, rows_total=800, seg_align=1,
             cap=0, ws=FAKE, ws_bytes=1 << 20)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INV), (dict(ids=None), INV), (dict(weights=None), INV), (dict(m_sizes=None), INV),
    (dict(row_of=None), INV), (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=65), INV),
    (dict(kind=2), INV), (dict(score=2), INV), (dict(rows_total=-1), INV), (dict(rows_total=1 << 31), INV),
    (dict(seg_align=0), INV), (dict(cap=-1), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=float("nan")), INV), (dict(scale=float("inf")), INV),
    (dict(n_groups=0), INV), (dict(n_groups=5), INV), (dict(n_groups=8, topk_groups=9), INV),
    (dict(n_groups=8, topk_groups=0), INV), (dict(group_top=0), INV), (dict(group_top=3), UNS),
    (dict(n_groups=128, E=128, k=1), UNS), (dict(E=1025), UNS), (dict(k=33), UNS), (dict(T=16773121), UNS),
    (dict(logits=ODD), INV), (dict(ids=ODD), INV), (dict(bias=ODD), INV), (dict(ws=None), WS), (dict(ws=EIGHT), WS),
    (dict(ws_bytes=8), WS),
])
def test_route_refusals(kw, status):
    assert call("moegg_route", ROUTE, kw) == status


def test_route_workspace_bytes():
    f = mg.lib().moegg_route_workspace_bytes
    assert f(-1, 8) == f(8, 0) == f(8, 1025) == f(1 << 30, 8) == 0
    assert f(0, 8) > 0 and f(1, 1) % 256 == 0
    assert f(4096, 64) == 256 * 64 * 2                     # 256 tiles of 16 tokens, 16-bit counts
    for E in (1, 63, 256, 1024):                           # a workspace for T tokens serves every smaller call
        sizes = [f(t, E) for t in [*range(5000), 16383, 65535, 65536, 1 << 20, 16773120]]
        assert sizes == sorted(sizes)
    assert [f(1100, e) for e in range(1, 1025)] == sorted(f(1100, e) for e in range(1, 1025))


RB = dict(logits=FAKE, kind=0, ids=FAKE, d_weights=FAKE, d_logits=FAKE, T=100, E=64, k=8, score=0, renorm=1, scale=1.0)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=None), INV), (dict(ids=None), INV), (dict(d_weights=None), INV), (dict(d_logits=None), INV),
    (dict(T=-1), INV), (dict(k=65), INV), (dict(kind=-1), INV), (dict(score=5), INV), (dict(scale=0.0), INV),
    (dict(E=2000), UNS), (dict(E=512, k=40), UNS), (dict(d_logits=ODD), INV),
])
def test_route_backward_refusals(kw, status):
    assert call("moegg_route_backward", RB, kw) == status


DISPATCH = dict(x=FAKE, row_of=FAKE, A=FAKE, A_scale=FAKE, T=100, k=8, K=256, rows=800, dtype=mg.FP8_E4M3)
PERMUTE_BAD = [
    (dict(T=-1), INV), (dict(k=0), INV), (dict(k=33), UNS), (dict(rows=-1), INV), (dict(rows=1 << 31), INV),
    (dict(row_of=None), INV), (dict(row_of=ODD), INV), (dict(T=1 << 26, k=32), UNS), (dict(T=1 << 25, k=1), UNS),
]


@pytest.mark.parametrize("kw,status", PERMUTE_BAD + [
    (dict(x=None), INV), (dict(A=None), INV), (dict(A_scale=None), INV), (dict(K=0), INV), (dict(K=200), UNS),
    (dict(dtype=9), INV), (dict(dtype=mg.FP8_E4M3_FP4_E2M1), INV), (dict(x=EIGHT), INV), (dict(A=EIGHT), INV),
    (dict(A_scale=ODD), INV), (dict(dtype=mg.BF16, x=ODD), INV),
])
def test_dispatch_refusals(kw, status):
    assert call("moegg_dispatch", DISPATCH, kw) == status


COMBINE = dict(Y=FAKE, row_of=FAKE, weights=FAKE, out=FAKE, T=100, k=8, N=256, rows=800)


@pytest.mark.parametrize("kw,status", PERMUTE_BAD + [
    (dict(Y=None), INV), (dict(out=None), INV), (dict(N=0), INV), (dict(Y=ODD), INV), (dict(weights=ODD), INV),
])
def test_combine_refusals(kw, status):
    assert call("moegg_combine", COMBINE, kw) == status


CB = dict(dout=FAKE, Y=FAKE, weights=FAKE, row_of=FAKE, dY=FAKE, dY_scale=FAKE, d_weights=FAKE, T=100, k=8, N=256,
          rows=800, dtype=mg.FP8_E4M3)


@pytest.mark.parametrize("kw,status", PERMUTE_BAD + [
    (dict(dout=None), INV), (dict(Y=None), INV), (dict(weights=None), INV), (dict(dY=None), INV),
    (dict(dY_scale=None), INV), (dict(d_weights=None), INV), (dict(N=100), UNS), (dict(dtype=-1), INV),
    (dict(dout=EIGHT), INV), (dict(Y=EIGHT), INV), (dict(dY=EIGHT), INV), (dict(d_weights=ODD), INV),
])
def test_combine_backward_refusals(kw, status):
    assert call("moegg_combine_backward", CB, kw) == status


CKPT_BAD = [(dict(m_sizes=None), INV), (dict(m_sizes=ODD), INV), (dict(G=0), INV), (dict(G=4097), INV),
            (dict(rows=-1), INV), (dict(rows=1 << 31), INV), (dict(I=0), INV), (dict(I=192), UNS),
            (dict(rows=1 << 30, I=1 << 20), UNS), (dict(I=1 << 22), UNS)]
FWD = dict(GU=FAKE, m_sizes=FAKE, H=FAKE, H_scale=FAKE, ckpt=FAKE, ckpt_scale=FAKE, G=8, rows=100, I=256,
           dtype=mg.FP8_E4M3)


@pytest.mark.parametrize("kw,status", CKPT_BAD + [
    (dict(GU=None), INV), (dict(H=None), INV), (dict(H_scale=None), INV), (dict(ckpt=None), INV),
    (dict(ckpt_scale=None), INV), (dict(GU=EIGHT), INV), (dict(ckpt=EIGHT), INV), (dict(H_scale=ODD), INV),
    (dict(dtype=mg.FP8_E4M3_E8M0), UNS), (dict(dtype=8), INV),
    (dict(rows=1 << 24, I=2048), UNS),                     # more work-items than a launch counts
])
def test_swiglu_checkpoint_refusals(kw, status):
    assert call("moegg_swiglu_checkpoint", FWD, kw) == status


BWD = dict(dH=FAKE, m_sizes=FAKE, ckpt=FAKE, ckpt_scale=FAKE, dGU=FAKE, H=FAKE, G=8, rows=100, I=256)


@pytest.mark.parametrize("kw,status", CKPT_BAD + [
    (dict(dH=None), INV), (dict(ckpt=None), INV), (dict(ckpt_scale=None), INV), (dict(dGU=None), INV),
    (dict(H=None), INV), (dict(dH=EIGHT), INV), (dict(H=EIGHT), INV),
])
def test_swiglu_checkpoint_backward_refusals(kw, status):
    assert call("moegg_swiglu_checkpoint_backward", BWD, kw) == status


BWD8 = dict(dH=FAKE, m_sizes=FAKE, ckpt=FAKE, ckpt_scale=FAKE, dGU=FAKE, dGU_scale=FAKE, dGU_k=FAKE, dGU_k_scale=FAKE,
            H_k=FAKE, H_k_scale=FAKE, G=8, rows=100, I=256, groups=9, dtype=mg.FP8_E4M3_SCALE_KM, k_e8m0=0)


@pytest.mark.parametrize("kw,status", CKPT_BAD + [(dict([(n, None)]), INV) for n in list(BWD8)[:10]] + [
    (dict(groups=-1), INV), (dict(dtype=mg.BF16), UNS), (dict(dtype=mg.FP8_E4M3_E8M0), UNS), (dict(dtype=6), INV),
    (dict(dGU_k=EIGHT), INV), (dict(H_k_scale=ODD), INV),
])
def test_swiglu_checkpoint_backward_fp8_refusals(kw, status):
    assert call("moegg_swiglu_checkpoint_backward_fp8", BWD8, kw) == status


KG = dict(X=FAKE, X_scale=FAKE, m_sizes=FAKE, X_k=FAKE, X_k_scale=FAKE, G=8, rows=100, I=512, groups=9,
          dtype=mg.FP8_E4M3, k_e8m0=0)


@pytest.mark.parametrize("kw,status", CKPT_BAD + [(dict([(n, None)]), INV) for n in list(KG)[:5]] + [
    (dict(I=384), UNS), (dict(groups=-1), INV), (dict(dtype=mg.FP8_E4M3_E8M0), UNS), (dict(X=EIGHT), INV),
    (dict(X_k=EIGHT), INV),
])
def test_checkpoint_to_k_groups_refusals(kw, status):
    assert call("moegg_checkpoint_to_k_groups", KG, kw) == status


# ------------------------------------------------------------------ the binding

def t(*shape, dtype=F32):
    return torch.zeros(*shape, dtype=dtype)


T, E, K_, R, W, S = 6, 16, 3, 20, 256, 4


def tensors(op):
    e4 = lambda *s: t(*s, dtype=U8).view(E4M3)               # noqa: E731
    if op == "route":
        return dict(logits=t(T, E), ids=t(T, K_, dtype=I32), weights=t(T, K_), m_sizes=t(E, dtype=I32),
                    row_of=t(T, K_, dtype=I32), ws=t(mg.route_workspace_bytes(T, E), dtype=U8), bias=t(E), rows_total=R)
    if op == "route_backward":
        return dict(logits=t(T, E, dtype=BF16), ids=t(T, K_, dtype=I32), d_weights=t(T, K_), d_logits=t(T, E, dtype=BF16))
    if op == "dispatch":
        return dict(x=t(T, W, dtype=BF16), row_of=t(T, K_, dtype=I32), A=e4(R, W), A_scale=t(R, W // 128))
    if op == "combine":
        return dict(Y=t(R, W, dtype=BF16), row_of=t(T, K_, dtype=I32), out=t(T, W, dtype=BF16), weights=t(T, K_))
    if op == "combine_backward":
        return dict(dout=t(T, W, dtype=BF16), Y=t(R, W, dtype=BF16), weights=t(T, K_), row_of=t(T, K_, dtype=I32),
                    dY=e4(R, W), d_weights=t(T, K_), dY_scale=t(W // 128, R), scale_km=True)
    if op == "swiglu_checkpoint":
        return dict(GU=t(R, 2 * W, dtype=BF16), m_sizes=t(5, dtype=I32), H=e4(R, W), ckpt=e4(R, 2 * W),
                    ckpt_scale=t(R, 2 * W // 128), H_scale=t(R, W // 128))
    if op == "swiglu_checkpoint_backward":
        return dict(dH=t(R, W, dtype=BF16), m_sizes=t(5, dtype=I32), ckpt=e4(R, 2 * W), ckpt_scale=t(R, 2 * W // 128),
                    dGU=t(R, 2 * W, dtype=BF16), H=t(R, W, dtype=BF16))
    if op == "swiglu_checkpoint_backward_fp8":
        return dict(dH=t(R, W, dtype=BF16), m_sizes=t(5, dtype=I32), ckpt=e4(R, 2 * W), ckpt_scale=t(R, 2 * W // 128),
                    dGU=e4(R, 2 * W), dGU_scale=t(R, 2 * W // 128), dGU_k=e4(R, 2 * W), dGU_k_scale=t(S, 2 * W),
                    H_k=e4(R, W), H_k_scale=t(S, W))
    return dict(X=e4(R, W), m_sizes=t(5, dtype=I32), X_k=e4(R, W), X_k_scale=t(S, W, dtype=U8), X_scale=t(R, W // 128))


OPS = ["route", "route_backward", "dispatch", "combine", "combine_backward", "swiglu_checkpoint",
       "swiglu_checkpoint_backward", "swiglu_checkpoint_backward_fp8", "checkpoint_to_k_groups"]


@pytest.mark.parametrize("op", OPS)
def test_correct_tensors_reach_the_device_check(op):
    with pytest.raises(ValueError, match="device tensor expected"):
        getattr(mg, op)(**tensors(op))


@pytest.mark.parametrize("op,name", [(op, n) for op in OPS for n, v in tensors(op).items()
                                     if isinstance(v, torch.Tensor)])
def test_each_tensor_is_checked(op, name):
    """A float64 tensor, a missing row or element, and one axis too many are refused by name."""
    good = tensors(op)[name]
    short = good.view(U8)[:-1].view(good.dtype) if good.dtype == E4M3 else good[:-1]
    leads = {"logits", "x", "out", "dout", "H", "dH", "X", "X_k_scale", "dGU_k_scale"}   # their first axis is the call's size
    for bad in [torch.zeros(good.shape, dtype=torch.float64), good[None, None]] + ([] if name in leads else [short]):
        if op == "combine" and name == "Y" and bad is short:
            continue                                       # the rows of Y are the call's rows
        if op == "swiglu_checkpoint_backward_fp8" and name == "m_sizes" or name == "m_sizes" and op != "route":
            if bad is short:
                continue                                   # any number of experts
        with pytest.raises(ValueError) as e:
            getattr(mg, op)(**{**tensors(op), name: bad})
        assert "device tensor" not in str(e.value), (op, name, e.value)


def test_missing_and_surplus_scales():
    a = tensors("dispatch")
    with pytest.raises(ValueError, match="A_scale"):
        mg.dispatch(**{**a, "A_scale": None})
    with pytest.raises(ValueError, match="A_scale: must be None"):
        mg.dispatch(**{**a, "A": t(R, W, dtype=BF16)})
    with pytest.raises(ValueError, match="A_scale: shape"):
        mg.dispatch(**a, scale_km=True)
    with pytest.raises(ValueError, match="scale_km"):
        mg.dispatch(**{**a, "A_scale": t(W // 128, R, dtype=U8)}, scale_km=True)
    with pytest.raises(ValueError, match="multiple of 128"):
        mg.dispatch(t(T, 200, dtype=BF16), a["row_of"], t(R, 200, dtype=U8).view(E4M3), t(R, 1))
    with pytest.raises(ValueError, match="fp32 scales expected"):
        f = tensors("swiglu_checkpoint")
        mg.swiglu_checkpoint(**{**f, "H_scale": t(W // 128, R, dtype=U8)})
    with pytest.raises(ValueError, match="H_k_scale: dtype"):
        f = tensors("swiglu_checkpoint_backward_fp8")
        mg.swiglu_checkpoint_backward_fp8(**{**f, "H_k_scale": t(S, W, dtype=U8)})


def test_small_route_workspace():
    a = tensors("route")
    with pytest.raises(ValueError, match="ws: 0 bytes"):
        mg.route(**{**a, "ws": a["ws"][:0]})


def test_native_tensor_checks_want_gpu_tensors():
    """The one-pass check answers None for whatever does not hold; the named checks follow it."""
    f = mg._args_module().pointers
    x = t(3, 4)
    assert f(()) == () and f((mg._ABSENT, mg._ABSENT)) == (None, None)
    for spec in [(x, "x", (3, 4), F32), (None, "x", (3, 4), F32), ([1.0], "x", (1,), F32), (x, "x", [3, 4], F32),
                 (x, "x", (3, 4), "float32"), (x, "x", (3, 4)), (x.to("meta"), "x", (3, 4), F32),
                 (x.to_sparse(), "x", (3, 4), F32)]:
        assert f((spec,)) is None and f((mg._ABSENT, spec)) is None
    assert f([mg._ABSENT]) is None
