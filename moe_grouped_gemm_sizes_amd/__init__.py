"""MI355X (gfx950) MoE grouped GEMM: a thin Python binding over libmoegg.so.

The binding only marshals arguments.  Every step of the grouped GEMM runs in
the HIP kernels behind the C ABI declared in include/moegg.h:
  - scheduler: counts -> padding accounting + tile list;
  - contiguous, masked and K-grouped GEMMs;
  - the layer around them: routing, token permutation, 8-bit activation checkpoints;
  - the block around that: RMS norm, the router's balance loss, low-rank adapters.
PyTorch supplies device memory and the current stream.  The layer calls check
their tensors in a native pass (csrc/args.cpp).  If the library has not been
built, `lib()` raises.  There is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.machinery
import importlib.util
import os
from dataclasses import dataclass
from typing import List, Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoegg.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "moegg.h")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_HIP = range(5)
BF16, FP8_E4M3, FP8_E4M3_E8M0, FP8_E4M3_FP4_E2M1, FP8_E4M3_SCALE_KM = 0, 1, 2, 3, 4
B_KN, B_NK, B_KN_PANEL, B_NK_PANEL = 0, 1, 2, 3
PANEL_CONTIGUOUS, PANEL_MASKED = 256, 128     # panel width P of the contiguous / SwiGLU and the masked calls
FLAG_NEGATIVE_COUNT, FLAG_ROWS_OVERFLOW, FLAG_COUNT_OVER_CAP, FLAG_BAD_EXEMPLAR = 0x1, 0x2, 0x4, 0x8
FLAG_SCALE_GROUPS = 0x10
FLAG_SYNC_TIMEOUT = 0x20
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1
LOGITS_FP32, LOGITS_BF16 = 0, 1
WEIGHT_FP32, WEIGHT_BF16 = 0, 1
Q_VALUES = (8, 16, 32, 64, 128, 256)
BLOCK_M_PER_EXPERT = -1          # per-expert tile heights (include/moegg.h)


class MoeggError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {lib().moegg_status_string(status).decode()} (status {status})")
        self.status = status


class _Stats(ctypes.Structure):
    _fields_ = [("U", ctypes.c_int64), ("P_exec", ctypes.c_int64), ("tiles", ctypes.c_int64),
                ("active", ctypes.c_int64), ("sum_sq", ctypes.c_int64), ("capacity_rows", ctypes.c_int64),
                ("P_at", ctypes.c_int64 * 6), ("block_m", ctypes.c_int32), ("error_flags", ctypes.c_uint32)]


class _Report(ctypes.Structure):
    _fields_ = [("effective_experts", ctypes.c_double), ("padding_fraction", ctypes.c_double * 6),
                ("useful_share", ctypes.c_double * 6), ("exec_padding_fraction", ctypes.c_double),
                ("physical_over_effective", ctypes.c_double)]


class _Tile(ctypes.Structure):
    _fields_ = [("expert", ctypes.c_int32), ("tile", ctypes.c_int32), ("row_start", ctypes.c_int32),
                ("rows_valid", ctypes.c_int32)]


@dataclass
class Stats:
    """Device-computed padding accounting of one scheduled call."""
    U: int
    P_exec: int
    tiles: int
    active: int
    sum_sq: int
    capacity_rows: int
    P_at: dict
    block_m: int
    error_flags: int

    def report(self) -> "Report":
        """The derived ratios, computed by the library (moegg_stats_report)."""
        st = _Stats(self.U, self.P_exec, self.tiles, self.active, self.sum_sq, self.capacity_rows,
                    (ctypes.c_int64 * 6)(*[self.P_at[q] for q in Q_VALUES]), self.block_m, self.error_flags)
        r = _Report()
        _check(lib().moegg_stats_report(ctypes.byref(st), ctypes.byref(r)), "moegg_stats_report")
        return Report(r.effective_experts, {q: r.padding_fraction[i] for i, q in enumerate(Q_VALUES)},
                      {q: r.useful_share[i] for i, q in enumerate(Q_VALUES)}, r.exec_padding_fraction,
                      r.physical_over_effective)

    @property
    def effective_experts(self) -> float:
        return self.report().effective_experts

    def padding_fraction(self, q: int) -> float:
        return self.report().padding_fraction[q]


@dataclass
class Report:
    """Ratios derived from Stats by the library: effective experts U^2 / sum m^2,
    padding fraction (P(q) - U) / P(q), useful share U / P(q), the executed rows'
    padding fraction and physical / effective work."""
    effective_experts: float
    padding_fraction: dict
    useful_share: dict
    exec_padding_fraction: float
    physical_over_effective: float


_lib = None
_VP, _I32, _I64, _SZ, _F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float

EXPORTS = {
    "moegg_version": (ctypes.c_int, []),
    "moegg_status_string": (ctypes.c_char_p, [_I32]),
    "moegg_workspace_bytes": (_SZ, [_I32, _I64]),
    "moegg_schedule": (_I32, [_VP, _I32, _I64, _I32, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_schedule_exemplar": (_I32, [_VP, _I32, _I64, _I32, _I32, _VP, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_selection_read": (_I32, [_VP, _VP, _VP]),
    "moegg_grouped_gemm_contiguous_scheduled": (_I32, [_VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I32,
                                                       _I32, _I32, _VP, _SZ, _VP]),
    "moegg_grouped_gemm_contiguous": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I32,
                                             _I32, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_grouped_gemm_contiguous_noalloc": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I32,
                                                     _I32, _I32, _I32, _VP]),
    "moegg_grouped_gemm_swiglu_scheduled": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I32,
                                                   _I32, _I32, _VP, _SZ, _VP]),
    "moegg_expert_mlp_fused": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32,
                                      _I32, _I32, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_grouped_gemm_masked": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32,
                                         _VP, _SZ, _VP]),
    "moegg_grouped_gemm_k_grouped": (_I32, [_VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_grouped_gemm_k_grouped_fp8": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I64,
                                                _VP, _SZ, _VP]),
    "moegg_grouped_gemm_k_grouped_e8m0": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _I64,
                                                 _VP, _SZ, _VP]),
    "moegg_route_workspace_bytes": (_SZ, [_I32, _I32]),
    "moegg_route": (_I32, [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _F32,
                           _I64, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_route_backward": (_I32, [_VP, _I32, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _F32, _VP]),
    "moegg_dispatch": (_I32, [_VP, _VP, _VP, _VP, _I32, _I32, _I32, _I64, _I32, _VP]),
    "moegg_combine": (_I32, [_VP, _VP, _VP, _VP, _I32, _I32, _I32, _I64, _VP]),
    "moegg_combine_backward": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I64, _I32, _VP]),
    "moegg_swiglu_checkpoint": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I32, _VP]),
    "moegg_swiglu_checkpoint_backward": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _VP]),
    "moegg_swiglu_checkpoint_backward_fp8": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I64,
                                                    _I32, _I64, _I32, _I32, _VP]),
    "moegg_checkpoint_to_k_groups": (_I32, [_VP, _VP, _VP, _VP, _VP, _I32, _I64, _I32, _I64, _I32, _I32, _VP]),
    "moegg_rms_norm": (_I32, [_VP, _VP, _VP, _I32, _F32, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _VP]),
    "moegg_rms_norm_workspace_bytes": (_SZ, [_I32, _I32]),
    "moegg_rms_norm_backward": (_I32, [_VP, _VP, _VP, _I32, _VP, _VP, _VP, _VP, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_balance_loss_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "moegg_balance_loss": (_I32, [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _VP, _SZ,
                                  _VP]),
    "moegg_balance_loss_backward": (_I32, [_VP, _I32, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _VP]),
    "moegg_lora_workspace_bytes": (_SZ, [_I32, _I32, _I32]),
    "moegg_lora": (_I32, [_VP, _VP, _VP, _VP, _VP, _VP, _VP, _I32, _I32, _I32, _I32, _I32, _VP, _SZ, _VP]),
    "moegg_stats_read": (_I32, [_VP, ctypes.POINTER(_Stats), _VP]),
    "moegg_stats_report": (_I32, [ctypes.POINTER(_Stats), ctypes.POINTER(_Report)]),
    "moegg_tile_list_read": (_I32, [_VP, ctypes.POINTER(_Tile), _I64, ctypes.POINTER(_I64), _VP]),
}


def lib():
    """The loaded HIP library.  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with python -m moe_grouped_gemm_sizes_amd.build")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("device tensor expected")
    if not t.is_contiguous():
        raise ValueError("contiguous tensor expected")
    return t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    # the handle alone: torch.cuda.current_stream() builds a Stream object, 2.8 us of a call's 10
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _check(status: int, what: str):
    if status != OK:
        raise MoeggError(status, what)


_E4M3 = torch.float8_e4m3fn


def _need(t: Optional[torch.Tensor], name: str, shape: Sequence[Optional[int]], dtypes):
    """ValueError unless `t` is a tensor of this shape (None matches any extent) and one of `dtypes`.
    The library sees only pointers, so every extent it will index is checked here."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: tensor expected")
    if t.dtype in dtypes and t.shape == tuple(shape):
        return
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != len(shape) or any(x is not None and d != x for d, x in zip(t.shape, shape)):
        want = "[" + ", ".join("*" if x is None else str(x) for x in shape) + "]"
        raise ValueError(f"{name}: shape {list(t.shape)}, expected {want}")


def _none(t, name: str, why: str):
    if t is not None:
        raise ValueError(f"{name}: must be None {why}")


def _one_device(*ts):
    first = None
    for t in ts:
        if isinstance(t, torch.Tensor):
            if first is None:
                first = t.get_device()
            elif t.get_device() != first:
                devs = {t.device for t in ts if isinstance(t, torch.Tensor)}
                raise ValueError(f"tensors on several devices: {sorted(str(d) for d in devs)}")


def _ws(ws, G: int, max_rows: int):
    _need(ws, "ws", [None], (torch.uint8,))
    # the library checks the byte count too; this names the problem
    need = workspace_bytes(G, max_rows)
    if ws.numel() < need:
        raise ValueError(f"ws: {ws.numel()} bytes, need {need} (workspace_bytes({G}, {max_rows}))")


def _counts(t, name: str, G: Optional[int] = None):
    _need(t, name, [G], (torch.int32,))
    if t.numel() < 1:
        raise ValueError(f"{name}: at least one expert expected")


def pack_panels(B: torch.Tensor, b_layout: int, P: int) -> torch.Tensor:
    """Weights [G, K, N] -> the paneled layout the kernels stream (include/moegg.h):
    B_KN_PANEL [G, N/P, K, P]; B_NK_PANEL [G, N/P, K/S, P, S] with S = 128 bytes of
    K.  Packed E2M1 weights (uint8) come as they are stored, [G, N, K/2], and go to
    B_NK_PANEL [G, N/P, K/128, P, 64].  P: PANEL_CONTIGUOUS for the contiguous and
    SwiGLU calls, PANEL_MASKED for the masked call.  A one-time weight transform."""
    if B.dtype == torch.uint8:
        if b_layout != B_NK_PANEL:
            raise ValueError("packed E2M1 weights have the B_NK_PANEL panel layout only")
        G, N, KB = B.shape
        if N % P or KB % 64:
            raise ValueError(f"[G, N, K/2] = {list(B.shape)}: N % {P} and K/2 % 64 must be 0")
        return B.reshape(G, N // P, P, KB // 64, 64).permute(0, 1, 3, 2, 4).contiguous()
    G, K, N = B.shape
    if N % P:
        raise ValueError(f"N = {N} is not a multiple of the panel width {P}")
    if b_layout == B_KN_PANEL:
        return B.reshape(G, K, N // P, P).permute(0, 2, 1, 3).contiguous()
    if b_layout == B_NK_PANEL:
        S = 128 // B.element_size()
        if K % S:
            raise ValueError(f"K = {K} is not a multiple of {S}")
        return B.reshape(G, K // S, S, N // P, P).permute(0, 3, 1, 4, 2).contiguous()
    raise ValueError(f"b_layout {b_layout} is not a panel layout")


def _weight_n(B, K: int, G: int, b_layout: int, P: int, dtypes) -> int:
    """N of weights B in layout b_layout, after checking B's shape against K and G."""
    if b_layout == B_KN:
        _need(B, "B", [G, K, None], dtypes)
        return B.shape[2]
    if b_layout == B_NK:
        _need(B, "B", [G, None, K], dtypes)
        return B.shape[1]
    if b_layout == B_KN_PANEL:
        _need(B, "B", [G, None, K, P], dtypes)
        return B.shape[1] * P
    if b_layout == B_NK_PANEL:
        S = 128 // B.element_size()
        _need(B, "B", [G, None, K // S, P, S], dtypes)
        if K % S:
            raise ValueError(f"K = {K}: the panel layout needs K % {S} == 0")
        return B.shape[1] * P
    raise ValueError(f"b_layout: {b_layout}")


def _operands(rows: int, K: int, A, A_scale, B, B_scale, G: int, b_layout: int, scale_km: bool,
              a_scale_rows_shape=None, P: int = PANEL_CONTIGUOUS) -> Tuple[int, int]:
    """Operand type code and N, after checking B, A_scale and B_scale against A's
    dtype, `rows` rows of K and G experts.  a_scale_rows_shape: the shape of a
    row-major fp32 activation-scale array ([rows, K/128] unless given).
    Formats (include/moegg.h): bf16 x bf16, no scales; e4m3 x e4m3 with fp32
    scales ([rows, K/128], or [K/128, rows] with scale_km) or E8M0 bytes
    ([K/128, rows]); e4m3 x packed E2M1 [G, N, K/2] (uint8) or its panels with E8M0
    bytes."""
    if b_layout not in (B_KN, B_NK, B_KN_PANEL, B_NK_PANEL):
        raise ValueError(f"b_layout: {b_layout}")
    if A.dtype == torch.bfloat16:
        _none(A_scale, "A_scale", "for bf16 operands")
        _none(B_scale, "B_scale", "for bf16 operands")
        if scale_km:
            raise ValueError("scale_km applies to e4m3 operands with fp32 scales")
        return BF16, _weight_n(B, K, G, b_layout, P, (torch.bfloat16,))
    if A.dtype != _E4M3:
        raise ValueError(f"A: bf16 or float8_e4m3fn expected, got {A.dtype}")
    if K % 128:
        raise ValueError(f"K = {K}: e4m3 operands need K % 128 == 0")
    if A_scale is None or B_scale is None:
        raise ValueError("e4m3 operands need A_scale and B_scale")
    if not isinstance(B, torch.Tensor):
        raise ValueError("B: tensor expected")
    if B.dtype == torch.uint8:                              # packed E2M1 weights [G, N, K/2] or its panels
        if b_layout == B_NK:
            N = B.shape[1]
            _need(B, "B", [G, N, K // 2], (torch.uint8,))
        elif b_layout == B_NK_PANEL:
            _need(B, "B", [G, None, K // 128, P, 64], (torch.uint8,))
            N = B.shape[1] * P
        else:
            raise ValueError("packed E2M1 weights are [G, N, K/2] (B_NK) or its panels (B_NK_PANEL)")
        _need(A_scale, "A_scale", [K // 128, rows], (torch.uint8,))
        _need(B_scale, "B_scale", [G, K // 128, N // 128], (torch.uint8,))
        if scale_km:
            raise ValueError("scale_km applies to e4m3 operands with fp32 scales")
        return FP8_E4M3_FP4_E2M1, N
    N = _weight_n(B, K, G, b_layout, P, (_E4M3,))
    if N % 128:
        raise ValueError(f"N = {N}: e4m3 operands need N % 128 == 0")
    if A_scale.dtype == torch.uint8:                        # E8M0 exponent bytes
        if scale_km:
            raise ValueError("scale_km applies to e4m3 operands with fp32 scales")
        _need(A_scale, "A_scale", [K // 128, rows], (torch.uint8,))
        _need(B_scale, "B_scale", [G, K // 128, N // 128], (torch.uint8,))
        return FP8_E4M3_E8M0, N
    if scale_km:
        _need(A_scale, "A_scale", [K // 128, rows], (torch.float32,))
    else:
        _need(A_scale, "A_scale", a_scale_rows_shape or [rows, K // 128], (torch.float32,))
    _need(B_scale, "B_scale", [G, K // 128, N // 128], (torch.float32,))
    return (FP8_E4M3_SCALE_KM if scale_km else FP8_E4M3), N


@functools.lru_cache(maxsize=64)
def workspace_bytes(G: int, max_rows: int) -> int:
    return int(lib().moegg_workspace_bytes(G, max_rows))


def workspace(G: int, max_rows: int, device="cuda") -> torch.Tensor:
    n = workspace_bytes(G, max_rows)
    if n == 0:
        raise ValueError("invalid workspace request")
    return torch.empty(n, dtype=torch.uint8, device=device)


def schedule(m_sizes: torch.Tensor, rows_total: int, ws: torch.Tensor, seg_align: int = 1, block_m: int = 0,
             N: int = 256, stream=None):
    _counts(m_sizes, "m_sizes")
    _ws(ws, m_sizes.numel(), rows_total)
    _one_device(m_sizes, ws)
    _check(lib().moegg_schedule(_p(m_sizes), m_sizes.numel(), rows_total, seg_align, block_m, N, _p(ws),
                                ws.numel(), _stream(stream)), "moegg_schedule")


EXEMPLAR_FIELDS = 10            # moegg_exemplar_t: size_class, lorenz[8], block_m (int32 each)
EXEMPLAR_TABLE_PATH = os.path.join(_HERE, "exemplars_mi355x.json")           # fp8 e4m3, fp32 block scales
EXEMPLAR_TABLE_PATHS = {"fp8": EXEMPLAR_TABLE_PATH, "bf16": os.path.join(_HERE, "exemplars_mi355x_bf16.json")}


def exemplar_table(device="cuda", path: Optional[str] = None, dtype: str = "fp8") -> torch.Tensor:
    """The exemplar table as an int32 [n, 10] device tensor (moegg_exemplar_t rows).
    Default: the table measured on MI355X for the operand type that ships with the
    package (dtype "fp8": e4m3 with fp32 block scales; "bf16")."""
    import json
    if path is None and dtype not in EXEMPLAR_TABLE_PATHS:
        raise ValueError(f"dtype: one of {sorted(EXEMPLAR_TABLE_PATHS)} expected, got {dtype!r}")
    with open(path or EXEMPLAR_TABLE_PATHS[dtype]) as f:
        rows = json.load(f)["exemplars"]
    t = torch.tensor([[r["size_class"], *r["lorenz"], r["block_m"]] for r in rows], dtype=torch.int32)
    return t.to(device)


def schedule_exemplar(m_sizes: torch.Tensor, rows_total: int, ws: torch.Tensor, exemplars: torch.Tensor,
                      hysteresis: int = 0, seg_align: int = 1, N: int = 256, stream=None):
    """moegg_schedule with the tile height matched to an exemplar on the device (see moegg.h)."""
    if exemplars.dtype != torch.int32 or exemplars.dim() != 2 or exemplars.shape[1] != EXEMPLAR_FIELDS:
        raise ValueError("exemplars: int32 [n, 10] expected")
    _counts(m_sizes, "m_sizes")
    _ws(ws, m_sizes.numel(), rows_total)
    _one_device(m_sizes, ws, exemplars)
    _check(lib().moegg_schedule_exemplar(_p(m_sizes), m_sizes.numel(), rows_total, seg_align, N, _p(exemplars),
                                         exemplars.shape[0], hysteresis, _p(ws), ws.numel(), _stream(stream)),
           "moegg_schedule_exemplar")


class _Selection(ctypes.Structure):
    _fields_ = [("exemplar", ctypes.c_int32), ("size_class", ctypes.c_int32), ("lorenz", ctypes.c_int32 * 8),
                ("distance", ctypes.c_int64)]


@dataclass
class Selection:
    exemplar: int
    size_class: int
    lorenz: Tuple[int, ...]
    distance: int


def selection_read(ws: torch.Tensor, stream=None) -> Selection:
    s = _Selection()
    _check(lib().moegg_selection_read(_p(ws), ctypes.c_void_p(ctypes.addressof(s)), _stream(stream)),
           "moegg_selection_read")
    return Selection(s.exemplar, s.size_class, tuple(s.lorenz), s.distance)


def grouped_gemm_contiguous_scheduled(A, B, C, G: int, ws, A_scale=None, B_scale=None, block_m: int = 0,
                                      b_layout: int = B_KN, stream=None, scale_km: bool = False):
    """The contiguous GEMM from the tile list already in ws (see moegg.h).
    scale_km: A_scale is fp32 [K/128, rows] (MOEGG_FP8_E4M3_SCALE_KM)."""
    _need(A, "A", [None, None], (torch.bfloat16, _E4M3))
    rows, K = A.shape
    code, N = _operands(rows, K, A, A_scale, B, B_scale, G, b_layout, scale_km)
    _need(C, "C", [rows, N], (torch.bfloat16,))
    _ws(ws, G, rows)
    _one_device(A, A_scale, B, B_scale, C, ws)
    _check(lib().moegg_grouped_gemm_contiguous_scheduled(
        _p(A), _p(A_scale), _p(B), _p(B_scale), _p(C), G, rows, K, N, code, b_layout,
        block_m, _p(ws), ws.numel(), _stream(stream)), "moegg_grouped_gemm_contiguous_scheduled")


def grouped_gemm_contiguous(A, B, C, m_sizes, ws, A_scale=None, B_scale=None, seg_align: int = 1,
                            block_m: int = 0, b_layout: int = B_KN, stream=None, scale_km: bool = False):
    """C[rows of expert e] = A[rows of expert e] @ B_e (see moegg.h).
    scale_km: A_scale is fp32 [K/128, rows] (MOEGG_FP8_E4M3_SCALE_KM)."""
    _counts(m_sizes, "m_sizes")
    G = m_sizes.numel()
    _need(A, "A", [None, None], (torch.bfloat16, _E4M3))
    rows, K = A.shape
    code, N = _operands(rows, K, A, A_scale, B, B_scale, G, b_layout, scale_km)
    _need(C, "C", [rows, N], (torch.bfloat16,))
    _ws(ws, G, rows)
    _one_device(A, A_scale, B, B_scale, C, m_sizes, ws)
    _check(lib().moegg_grouped_gemm_contiguous(
        _p(A), _p(A_scale), _p(B), _p(B_scale), _p(C), _p(m_sizes), G, rows, K, N,
        seg_align, code, b_layout, block_m, _p(ws), ws.numel(), _stream(stream)),
        "moegg_grouped_gemm_contiguous")


NOALLOC_SCRATCH_BYTES = 1 << 20          # MOEGG_NOALLOC_SCRATCH_BYTES


def grouped_gemm_contiguous_noalloc(A, B, C, m_sizes, A_scale=None, B_scale=None, seg_align: int = 1,
                                    block_m: int = 0, b_layout: int = B_KN, stream=None, scale_km: bool = False):
    """grouped_gemm_contiguous without a workspace: the library's fixed per-GPU
    scratch array holds the schedule (see moegg.h); nothing is allocated."""
    _counts(m_sizes, "m_sizes")
    G = m_sizes.numel()
    _need(A, "A", [None, None], (torch.bfloat16, _E4M3))
    rows, K = A.shape
    code, N = _operands(rows, K, A, A_scale, B, B_scale, G, b_layout, scale_km)
    _need(C, "C", [rows, N], (torch.bfloat16,))
    _one_device(A, A_scale, B, B_scale, C, m_sizes)
    _check(lib().moegg_grouped_gemm_contiguous_noalloc(
        _p(A), _p(A_scale), _p(B), _p(B_scale), _p(C), _p(m_sizes), G, rows, K, N,
        seg_align, code, b_layout, block_m, _stream(stream)), "moegg_grouped_gemm_contiguous_noalloc")


def interleave_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor) -> torch.Tensor:
    """Gate and up weights [G, I, K] (K-contiguous) -> W1 [G, 2I, K] in the row
    order moegg_grouped_gemm_swiglu_scheduled takes: 16 gate rows, then the 16
    up rows of the same outputs.  A one-time weight transform."""
    G, I, K = w_gate.shape
    if w_up.shape != w_gate.shape or I % 16:
        raise ValueError("gate and up weights [G, I, K] with I % 16 == 0 expected")
    return torch.stack([w_gate.reshape(G, I // 16, 16, K), w_up.reshape(G, I // 16, 16, K)], dim=2) \
        .reshape(G, 2 * I, K).contiguous()


def grouped_gemm_swiglu_scheduled(A, W1, H, G: int, ws, A_scale=None, W1_scale=None, block_m: int = 0,
                                  H_scale=None, stream=None, scale_km: bool = False, b_layout: int = B_NK):
    """H = silu(A W_gate) * (A W_up) per expert, from the tile list in ws (see moegg.h).
    H bf16 [rows, I]; or, with H_scale (fp32 [rows, I/128]), H float8_e4m3fn codes.
    scale_km: A_scale fp32 [K/128, rows] in, H_scale [I/128, rows] out."""
    _need(A, "A", [None, None], (torch.bfloat16, _E4M3))
    rows, K = A.shape
    if b_layout not in (B_NK, B_NK_PANEL):
        raise ValueError("W1: [G, 2I, K] (B_NK) or its panels (B_NK_PANEL)")
    code, N = _operands(rows, K, A, A_scale, W1, W1_scale, G, b_layout, scale_km)
    if N % 256:
        raise ValueError(f"W1: {N} interleaved gate/up rows, a multiple of 256 expected")
    I = N // 2
    if H_scale is None:
        _need(H, "H", [rows, I], (torch.bfloat16,))
    else:
        _need(H, "H", [rows, I], (_E4M3,))
        _need(H_scale, "H_scale", [I // 128, rows] if scale_km else [rows, I // 128], (torch.float32,))
    _ws(ws, G, rows)
    _one_device(A, A_scale, W1, W1_scale, H, H_scale, ws)
    _check(lib().moegg_grouped_gemm_swiglu_scheduled(
        _p(A), _p(A_scale), _p(W1), _p(W1_scale), _p(H), _p(H_scale), G, rows, K, I, code,
        b_layout, block_m, _p(ws), ws.numel(), _stream(stream)), "moegg_grouped_gemm_swiglu_scheduled")


def expert_mlp_fused(A, W1, W2, H, Y, m_sizes, ws, A_scale, W1_scale, W2_scale, H_scale, seg_align: int = 1,
                     b_layout: int = B_NK, scale_km: bool = False, stream=None):
    """Y = SwiGLU(A W1) W2 per expert in one launch (see moegg.h): e4m3 A [rows, K], W1
    [G, 2I, K] (gate/up interleaved), W2 [G, N2, I], fp32 scales; H e4m3 [rows, I] with H_scale the
    caller's intermediate, written and read back by the kernel; Y bf16 [rows, N2].  b_layout B_NK or
    B_NK_PANEL (P = PANEL_CONTIGUOUS) for both weights; scale_km: A_scale [K/128, rows] in and
    H_scale [I/128, rows]."""
    _need(A, "A", [None, None], (_E4M3,))
    rows, K = A.shape
    if b_layout not in (B_NK, B_NK_PANEL):
        raise ValueError("W1, W2: [G, N, K] (B_NK) or its panels (B_NK_PANEL)")
    _counts(m_sizes, "m_sizes")
    G = m_sizes.numel()
    code, N = _operands(rows, K, A, A_scale, W1, W1_scale, G, b_layout, scale_km)
    if N % 256:
        raise ValueError(f"W1: {N} interleaved gate/up rows, a multiple of 256 expected")
    I = N // 2
    _need(H, "H", [rows, I], (_E4M3,))
    _need(H_scale, "H_scale", [I // 128, rows] if scale_km else [rows, I // 128], (torch.float32,))
    code2, N2 = _operands(rows, I, H, H_scale, W2, W2_scale, G, b_layout, scale_km)
    if code2 != code or N2 % 256:
        raise ValueError(f"W2: e4m3 [G, N2, I] with N2 % 256 == 0 expected, got N2 = {N2}")
    _need(Y, "Y", [rows, N2], (torch.bfloat16,))
    _ws(ws, G, rows)
    _one_device(A, A_scale, W1, W1_scale, W2, W2_scale, H, H_scale, Y, m_sizes, ws)
    _check(lib().moegg_expert_mlp_fused(
        _p(A), _p(A_scale), _p(W1), _p(W1_scale), _p(W2), _p(W2_scale), _p(H), _p(H_scale), _p(Y),
        _p(m_sizes), G, rows, K, I, N2, seg_align, code, b_layout, _p(ws), ws.numel(), _stream(stream)),
        "moegg_expert_mlp_fused")


def grouped_gemm_masked(A, B, C, masked_m, ws=None, A_scale=None, B_scale=None, b_layout: int = B_KN,
                        stream=None, scale_km: bool = False):
    """C[e, r] = A[e, r] @ B_e for r < masked_m[e] (see moegg.h).
    scale_km: A_scale is fp32 [K/128, G * cap] (MOEGG_FP8_E4M3_SCALE_KM)."""
    _need(A, "A", [None, None, None], (torch.bfloat16, _E4M3))
    G, cap, K = A.shape
    _counts(masked_m, "masked_m", G)
    code, N = _operands(G * cap, K, A, A_scale, B, B_scale, G, b_layout, scale_km,
                        a_scale_rows_shape=[G, cap, K // 128], P=PANEL_MASKED)
    _need(C, "C", [G, cap, N], (torch.bfloat16,))
    if ws is not None:
        _ws(ws, G, G * cap)
    _one_device(A, A_scale, B, B_scale, C, masked_m, ws)
    _check(lib().moegg_grouped_gemm_masked(
        _p(A), _p(A_scale), _p(B), _p(B_scale), _p(C), _p(masked_m), G, cap, K, N, code, b_layout,
        _p(ws), 0 if ws is None else ws.numel(), _stream(stream)), "moegg_grouped_gemm_masked")


def k_scale_groups(t_sizes: Sequence[int]) -> int:
    """Rows the K-grouped fp8 scale arrays need: sum over experts of ceil(t_e / 128)."""
    return sum((max(int(t), 0) + 127) // 128 for t in t_sizes)


def grouped_gemm_k_grouped(X, dY, dW, t_sizes, ws, X_scale=None, dY_scale=None, stream=None):
    """dW[e] = X_e^T @ dY_e over expert e's rows (see moegg.h).  bf16 X and dY;
    or e4m3 X and dY with scales X_scale [S, Mw], dY_scale [S, Nw], one row per
    128-row group of each expert's segment (k_scale_groups gives S): fp32, or
    uint8 E8M0 exponent bytes (2^(b - 127))."""
    _counts(t_sizes, "t_sizes")
    G = t_sizes.numel()
    _need(X, "X", [None, None], (torch.bfloat16, _E4M3))
    T, Mw = X.shape
    _need(dY, "dY", [T, None], (X.dtype,))
    Nw = dY.shape[1]
    _need(dW, "dW", [G, Mw, Nw], (torch.float32,))
    _ws(ws, G, 0)
    if X.dtype == torch.bfloat16:
        _none(X_scale, "X_scale", "for bf16 operands")
        _none(dY_scale, "dY_scale", "for bf16 operands")
        _one_device(X, dY, dW, t_sizes, ws)
        _check(lib().moegg_grouped_gemm_k_grouped(
            _p(X), _p(dY), _p(dW), _p(t_sizes), G, T, Mw, Nw, _p(ws), ws.numel(), _stream(stream)),
            "moegg_grouped_gemm_k_grouped")
        return
    _need(X_scale, "X_scale", [None, Mw], (torch.float32, torch.uint8))
    S = X_scale.shape[0]
    _need(dY_scale, "dY_scale", [S, Nw], (X_scale.dtype,))
    _one_device(X, X_scale, dY, dY_scale, dW, t_sizes, ws)
    if X_scale.dtype == torch.uint8:
        _check(lib().moegg_grouped_gemm_k_grouped_e8m0(
            _p(X), _p(X_scale), _p(dY), _p(dY_scale), _p(dW), _p(t_sizes), G, T, Mw, Nw, S, _p(ws), ws.numel(),
            _stream(stream)), "moegg_grouped_gemm_k_grouped_e8m0")
        return
    _check(lib().moegg_grouped_gemm_k_grouped_fp8(
        _p(X), _p(X_scale), _p(dY), _p(dY_scale), _p(dW), _p(t_sizes), G, T, Mw, Nw, S, _p(ws), ws.numel(),
        _stream(stream)), "moegg_grouped_gemm_k_grouped_fp8")


# ---------------------------------------------------------------- the layer around the grouped GEMMs


@functools.lru_cache(maxsize=4096)
def route_workspace_bytes(T: int, E: int) -> int:
    return int(lib().moegg_route_workspace_bytes(T, E))


def route_workspace(T: int, E: int, device="cuda") -> torch.Tensor:
    n = route_workspace_bytes(T, E)
    if n == 0:
        raise ValueError("invalid workspace request")
    return torch.empty(n, dtype=torch.uint8, device=device)


_ABSENT = (None, "", None, None)                             # an optional tensor that was not given


def _args_module():
    """The tensor checks of csrc/args.cpp.  Raises if they have not been built."""
    global _args
    if _args is None:
        path = os.path.join(_HERE, "_args.so")
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with python -m moe_grouped_gemm_sizes_amd.build")
        loader = importlib.machinery.ExtensionFileLoader("_args", path)
        _args = importlib.util.module_from_spec(importlib.util.spec_from_loader("_args", loader))
        loader.exec_module(_args)
    return _args


_args = None


def _pointers(*specs):
    """Data pointers of (tensor, name, shape, dtype) specs; None for _ABSENT.  One native pass where each is a
    contiguous tensor as specified on one GPU; else the checks one by one, for their messages."""
    out = (_args or _args_module()).pointers(specs)
    if out is not None:
        return out
    for t, name, shape, dtype in specs:
        if shape is not None:
            _need(t, name, shape, (dtype,))
    _one_device(*(s[0] for s in specs))
    return [_p(s[0]) for s in specs]


def _matrix(t, name: str, dtypes):
    """Shape of a matrix of one of `dtypes`."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes:
        shape = t.shape
        if len(shape) == 2:
            return shape
    _need(t, name, (None, None), dtypes)


_F, _H, _I = torch.float32, torch.bfloat16, torch.int32


def route(logits, ids, weights, m_sizes, row_of, ws, *, rows_total: int, bias=None, score: int = SCORE_SOFTMAX,
          n_groups: int = 1, topk_groups: int = 1, group_top: int = 1, renorm: bool = True, scale: float = 1.0,
          seg_align: int = 1, cap: int = 0, stream=None):
    """logits [T, E] -> ids, weights, row_of [T, k] and m_sizes [E] (see moegg.h): top-k experts by softmax or
    sigmoid score (plus bias [E] for the choice alone), group-limited when n_groups > 1; row_of is the row of every
    assignment in the contiguous layout of rows_total rows, or with cap > 0 in [E, cap] capacity buffers
    (rows_total = E * cap); -1 where there is none.  ws: route_workspace(T, E), or of more tokens or experts."""
    T, E = _matrix(logits, "logits", (_F, _H))
    k = _matrix(ids, "ids", (_I,))[1]
    kind = logits.dtype
    n = ws.numel() if isinstance(ws, torch.Tensor) else 0
    need = route_workspace_bytes(T, E)
    if n < need:
        raise ValueError(f"ws: {n} bytes, need {need} (route_workspace_bytes({T}, {E}))")
    l, i, w, m, r, b, s = _pointers(
        (logits, "logits", (T, E), kind), (ids, "ids", (T, k), _I), (weights, "weights", (T, k), _F),
        (m_sizes, "m_sizes", (E,), _I), (row_of, "row_of", (T, k), _I), (bias, "bias", (E,), _F) if bias is not None else _ABSENT,
        (ws, "ws", (n,), torch.uint8))
    _check(lib().moegg_route(l, LOGITS_BF16 if kind is _H else LOGITS_FP32, b, i, w, m, r, T, E, k, score, n_groups,
                             topk_groups, group_top, renorm, scale, rows_total, seg_align, cap, s, n,
                             _stream(stream)), "moegg_route")


def route_backward(logits, ids, d_weights, d_logits, *, score: int = SCORE_SOFTMAX, renorm: bool = True,
                   scale: float = 1.0, stream=None):
    """d_logits [T, E] (logits' dtype) from d_weights [T, k] and the ids that route chose (see moegg.h)."""
    T, E = _matrix(logits, "logits", (_F, _H))
    k = _matrix(ids, "ids", (_I,))[1]
    kind = logits.dtype
    l, i, dw, dl = _pointers((logits, "logits", (T, E), kind), (ids, "ids", (T, k), _I),
                             (d_weights, "d_weights", (T, k), _F), (d_logits, "d_logits", (T, E), kind))
    _check(lib().moegg_route_backward(l, LOGITS_BF16 if kind is _H else LOGITS_FP32, i, dw, dl, T, E, k, score, renorm,
                                      scale, _stream(stream)), "moegg_route_backward")


def _row_operand(A, name: str, A_scale, width: int, scale_km: bool):
    """Rows and operand type code of an expert-side operand [rows, width] or [G, cap, width], and the specs of it and
    its scales."""
    if not isinstance(A, torch.Tensor) or A.dim() not in (2, 3):
        raise ValueError(f"{name}: tensor [rows, width] or [G, cap, width] expected")
    kind, lead = A.dtype, A.shape[:-1]
    rows = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    spec = (A, name, lead + (width,), kind)
    if kind is _H:
        _none(A_scale, f"{name}_scale", "for a bf16 operand")
        if scale_km:
            raise ValueError("scale_km applies to e4m3 operands with fp32 scales")
        return rows, BF16, spec, _ABSENT
    if kind is not _E4M3:
        _need(A, name, lead + (width,), (_H, _E4M3))
    if width % 128:
        raise ValueError(f"{name}: width {width}, e4m3 operands need a multiple of 128")
    groups = width // 128
    if isinstance(A_scale, torch.Tensor) and A_scale.dtype is torch.uint8:
        if scale_km:
            raise ValueError("scale_km applies to e4m3 operands with fp32 scales")
        return rows, FP8_E4M3_E8M0, spec, (A_scale, f"{name}_scale", (groups, rows), torch.uint8)
    return (rows, FP8_E4M3_SCALE_KM if scale_km else FP8_E4M3, spec,
            (A_scale, f"{name}_scale", (groups, rows) if scale_km else lead + (groups,), _F))


def dispatch(x, row_of, A, A_scale=None, *, scale_km: bool = False, stream=None):
    """A[row_of[t, j]] = x[t] (see moegg.h).  x bf16 [T, K]; A bf16 or e4m3, [rows, K] or [G, cap, K], with the
    scales of the grouped GEMM that reads it: fp32 [rows, K/128] ([G, cap, K/128]), [K/128, rows] (scale_km), or
    uint8 E8M0 bytes [K/128, rows]."""
    T, K = _matrix(x, "x", (_H,))
    k = _matrix(row_of, "row_of", (_I,))[1]
    rows, code, spec, spec_scale = _row_operand(A, "A", A_scale, K, scale_km)
    px, pr, pa, ps = _pointers((x, "x", (T, K), _H), (row_of, "row_of", (T, k), _I), spec, spec_scale)
    _check(lib().moegg_dispatch(px, pr, pa, ps, T, k, K, rows, code, _stream(stream)), "moegg_dispatch")


def _expert_rows(Y, N: int):
    """Rows of bf16 Y [rows, N] or [G, cap, N], and its spec."""
    if not isinstance(Y, torch.Tensor) or Y.dim() not in (2, 3):
        raise ValueError("Y: tensor [rows, N] or [G, cap, N] expected")
    lead = Y.shape[:-1]
    return lead[0] if len(lead) == 1 else lead[0] * lead[1], (Y, "Y", lead + (N,), _H)


def combine(Y, row_of, out, weights=None, *, stream=None):
    """out[t] = sum_j weights[t, j] * Y[row_of[t, j]] (see moegg.h); weights None: all 1, which is also dispatch's
    backward pass.  Y bf16 [rows, N] or [G, cap, N], out bf16 [T, N], weights fp32 [T, k]."""
    T, N = _matrix(out, "out", (_H,))
    k = _matrix(row_of, "row_of", (_I,))[1]
    rows, spec = _expert_rows(Y, N)
    py, pr, po, pw = _pointers(spec, (row_of, "row_of", (T, k), _I), (out, "out", (T, N), _H),
                               (weights, "weights", (T, k), _F) if weights is not None else _ABSENT)
    _check(lib().moegg_combine(py, pr, pw, po, T, k, N, rows, _stream(stream)), "moegg_combine")


def combine_backward(dout, Y, weights, row_of, dY, d_weights, dY_scale=None, *, scale_km: bool = False, stream=None):
    """dY[row_of[t, j]] = weights[t, j] * dout[t] in dY's operand format (as dispatch's A), and d_weights[t, j] =
    <Y[row_of[t, j]], dout[t]> (see moegg.h)."""
    T, N = _matrix(dout, "dout", (_H,))
    k = _matrix(row_of, "row_of", (_I,))[1]
    rows, code, spec, spec_scale = _row_operand(dY, "dY", dY_scale, N, scale_km)
    y_rows, y_spec = _expert_rows(Y, N)
    if y_rows != rows:
        raise ValueError(f"Y: shape {list(Y.shape)}, expected {rows} rows as dY")
    pd, py, pw, pr, pg, ps, pdw = _pointers(
        (dout, "dout", (T, N), _H), y_spec, (weights, "weights", (T, k), _F), (row_of, "row_of", (T, k), _I), spec,
        spec_scale, (d_weights, "d_weights", (T, k), _F))
    _check(lib().moegg_combine_backward(pd, py, pw, pr, pg, ps, pdw, T, k, N, rows, code, _stream(stream)),
           "moegg_combine_backward")


def _no_e8m0(code: int, name: str):
    if code == FP8_E4M3_E8M0:
        raise ValueError(f"{name}: fp32 scales expected")


def _token_group_scales(X_scale, name: str) -> int:
    return _matrix(X_scale, name, (_F, torch.uint8))[0]


def _counts_spec(m_sizes):
    """The number of experts, and m_sizes' spec."""
    if not isinstance(m_sizes, torch.Tensor) or m_sizes.dim() != 1 or m_sizes.shape[0] < 1:
        _counts(m_sizes, "m_sizes")
    G = m_sizes.shape[0]
    return G, (m_sizes, "m_sizes", (G,), _I)


def swiglu_checkpoint(GU, m_sizes, H, ckpt, ckpt_scale, H_scale=None, *, scale_km: bool = False, stream=None):
    """H = silu(g) * u of GU bf16 [rows, 2I] (columns in interleave_gate_up's order), and GU kept as e4m3 ckpt
    [rows, 2I] with fp32 ckpt_scale [rows, 2I/128] (see moegg.h).  H bf16 [rows, I], or e4m3 with H_scale fp32
    [rows, I/128] ([I/128, rows] with scale_km)."""
    rows, I = _matrix(H, "H", (_H, _E4M3))
    _, code, spec, spec_scale = _row_operand(H, "H", H_scale, I, scale_km)
    _no_e8m0(code, "H_scale")
    G, counts = _counts_spec(m_sizes)
    pg, pm, ph, phs, pc, pcs = _pointers(
        (GU, "GU", (rows, 2 * I), _H), counts, spec, spec_scale, (ckpt, "ckpt", (rows, 2 * I), _E4M3),
        (ckpt_scale, "ckpt_scale", (rows, 2 * I // 128), _F))
    _check(lib().moegg_swiglu_checkpoint(pg, pm, ph, phs, pc, pcs, G, rows, I, code, _stream(stream)),
           "moegg_swiglu_checkpoint")


def swiglu_checkpoint_backward(dH, m_sizes, ckpt, ckpt_scale, dGU, H, *, stream=None):
    """dGU bf16 [rows, 2I] and H bf16 [rows, I] again, from dH bf16 [rows, I] and the checkpoint (see moegg.h)."""
    rows, I = _matrix(dH, "dH", (_H,))
    G, counts = _counts_spec(m_sizes)
    pd, pm, pc, pcs, pg, ph = _pointers(
        (dH, "dH", (rows, I), _H), counts, (ckpt, "ckpt", (rows, 2 * I), _E4M3),
        (ckpt_scale, "ckpt_scale", (rows, 2 * I // 128), _F), (dGU, "dGU", (rows, 2 * I), _H), (H, "H", (rows, I), _H))
    _check(lib().moegg_swiglu_checkpoint_backward(pd, pm, pc, pcs, pg, ph, G, rows, I, _stream(stream)),
           "moegg_swiglu_checkpoint_backward")


def swiglu_checkpoint_backward_fp8(dH, m_sizes, ckpt, ckpt_scale, dGU, dGU_scale, dGU_k, dGU_k_scale, H_k, H_k_scale,
                                   *, scale_km: bool = False, stream=None):
    """The operands of both gradients' products from dH bf16 [rows, I] and the checkpoint (see moegg.h): dGU e4m3
    [rows, 2I] with fp32 dGU_scale [rows, 2I/128] ([2I/128, rows] with scale_km); dGU_k e4m3 [rows, 2I] and H_k
    e4m3 [rows, I] with scales per token group, [S, 2I] and [S, I], fp32 or uint8 E8M0 bytes (k_scale_groups)."""
    rows, I = _matrix(dH, "dH", (_H,))
    _need(dGU, "dGU", (rows, 2 * I), (_E4M3,))
    _, code, spec, spec_scale = _row_operand(dGU, "dGU", dGU_scale, 2 * I, scale_km)
    _no_e8m0(code, "dGU_scale")
    G, counts = _counts_spec(m_sizes)
    S = _token_group_scales(dGU_k_scale, "dGU_k_scale")
    kind = dGU_k_scale.dtype
    p = _pointers(
        (dH, "dH", (rows, I), _H), counts, (ckpt, "ckpt", (rows, 2 * I), _E4M3),
        (ckpt_scale, "ckpt_scale", (rows, 2 * I // 128), _F), spec, spec_scale,
        (dGU_k, "dGU_k", (rows, 2 * I), _E4M3), (dGU_k_scale, "dGU_k_scale", (S, 2 * I), kind),
        (H_k, "H_k", (rows, I), _E4M3), (H_k_scale, "H_k_scale", (S, I), kind))
    _check(lib().moegg_swiglu_checkpoint_backward_fp8(*p, G, rows, I, S, code, kind is torch.uint8, _stream(stream)),
           "moegg_swiglu_checkpoint_backward_fp8")


def checkpoint_to_k_groups(X, m_sizes, X_k, X_k_scale, X_scale=None, *, scale_km: bool = False, stream=None):
    """A saved activation X [rows, M] (bf16, or e4m3 with fp32 scales [rows, M/128], [M/128, rows] with scale_km) as
    an operand of grouped_gemm_k_grouped: X_k e4m3 [rows, M] with X_k_scale [S, M], fp32 or uint8 E8M0 (see moegg.h)."""
    rows, M = _matrix(X, "X", (_H, _E4M3))
    _, code, spec, spec_scale = _row_operand(X, "X", X_scale, M, scale_km)
    _no_e8m0(code, "X_scale")
    G, counts = _counts_spec(m_sizes)
    S = _token_group_scales(X_k_scale, "X_k_scale")
    kind = X_k_scale.dtype
    px, ps, pm, pk, pks = _pointers(spec, spec_scale, counts, (X_k, "X_k", (rows, M), _E4M3),
                                    (X_k_scale, "X_k_scale", (S, M), kind))
    _check(lib().moegg_checkpoint_to_k_groups(px, ps, pm, pk, pks, G, rows, M, S, code, kind is torch.uint8,
                                              _stream(stream)), "moegg_checkpoint_to_k_groups")


# ---------------------------------------------------------------- the block around the layer


def _workspace_of(n: int, device) -> torch.Tensor:
    if n == 0:
        raise ValueError("invalid workspace request")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _ws_spec(ws, need: int, what: str):
    """ws' size in bytes, and its spec."""
    n = ws.numel() if isinstance(ws, torch.Tensor) else 0
    if n < need:
        raise ValueError(f"ws: {n} bytes, need {need} ({what})")
    return n, (ws, "ws", (n,), torch.uint8)


def _stream_for(t, stream):
    """The stream of a call on t's device, which has to be the current one unless a stream of it is given: launches go
    to the stream's device, those of a default stream (handle 0) to the current one."""
    if stream is not None:
        if stream.device_index != t.get_device():
            raise ValueError(f"tensors on cuda:{t.get_device()}, stream of cuda:{stream.device_index}")
        if stream.cuda_stream == 0 and torch._C._cuda_getDevice() != t.get_device():
            raise ValueError(f"default stream of cuda:{t.get_device()}, the current device is another")
        return stream.cuda_stream
    current = torch.cuda.current_device()
    if t.get_device() != current:
        raise ValueError(f"tensors on cuda:{t.get_device()}, the current device is cuda:{current}")
    return torch._C._cuda_getCurrentRawStream(current)


def _optional(t, name: str, shape, kind):
    return (t, name, shape, kind) if t is not None else _ABSENT


def _norm_weight(weight, K: int):
    """Type code of a norm's weight, and its spec."""
    kind = weight.dtype if isinstance(weight, torch.Tensor) else None
    if kind is not _H and kind is not _F:
        _need(weight, "weight", (K,), (_F, _H))
    return WEIGHT_BF16 if kind is _H else WEIGHT_FP32, (weight, "weight", (K,), kind)


def rms_norm(x, weight, *, y=None, q=None, q_scale=None, residual=None, sum_out=None, rstd=None, eps: float = 1e-6,
             scale_km: bool = False, stream=None):
    """h = x + residual (bf16, to sum_out), then h * rstd * weight with rstd = 1 / sqrt(mean h^2 + eps) (see moegg.h):
    as y bf16 [T, K], and as q e4m3 [T, K] with the scales of the grouped GEMM that reads it: fp32 [T, K/128],
    [K/128, T] (scale_km), or uint8 E8M0 bytes [K/128, T].  x, residual, sum_out bf16 [T, K]; weight fp32 or bf16 [K];
    rstd fp32 [T].  y or q, or both; sum_out may be x or residual."""
    T, K = _matrix(x, "x", (_H,))
    weight_kind, weight_spec = _norm_weight(weight, K)
    if q is None:
        _none(q_scale, "q_scale", "without q")
        if y is None:
            raise ValueError("y or q expected")
        if scale_km:
            raise ValueError("scale_km applies to e4m3 operands with fp32 scales")
        code, q_spec, scale_spec = BF16, _ABSENT, _ABSENT
    else:
        if _matrix(q, "q", (_E4M3,)) != (T, K):
            _need(q, "q", (T, K), (_E4M3,))
        _, code, q_spec, scale_spec = _row_operand(q, "q", q_scale, K, scale_km)
    if residual is None:
        _none(sum_out, "sum_out", "without a residual")
    px, pr, pw, ps, py, pq, pqs, pd = _pointers(
        (x, "x", (T, K), _H), _optional(residual, "residual", (T, K), _H), weight_spec,
        _optional(sum_out, "sum_out", (T, K), _H), _optional(y, "y", (T, K), _H), q_spec, scale_spec,
        _optional(rstd, "rstd", (T,), _F))
    _check(lib().moegg_rms_norm(px, pr, pw, weight_kind, eps, ps, py, pq, pqs, pd, T, K, code, _stream_for(x, stream)),
           "moegg_rms_norm")


@functools.lru_cache(maxsize=4096)
def rms_norm_workspace_bytes(T: int, K: int) -> int:
    return int(lib().moegg_rms_norm_workspace_bytes(T, K))


def rms_norm_workspace(T: int, K: int, device="cuda") -> torch.Tensor:
    return _workspace_of(rms_norm_workspace_bytes(T, K), device)


def rms_norm_backward(dy, h, weight, rstd, dx, d_weight=None, ws=None, *, d_sum=None, stream=None):
    """dx bf16 [T, K], the gradient of x and of the residual, and d_weight fp32 [K] (None: left out) from dy bf16 [T, K]
    (see moegg.h); h is rms_norm's sum_out (or x), rstd as it wrote it, d_sum bf16 [T, K] the gradient that arrives at
    the sum itself.  ws: rms_norm_workspace(T, K), or of more tokens; needed for d_weight.  dx may be dy, h or d_sum."""
    T, K = _matrix(dy, "dy", (_H,))
    weight_kind, weight_spec = _norm_weight(weight, K)
    n, ws_spec = 0, _ABSENT
    if d_weight is not None:
        n, ws_spec = _ws_spec(ws, rms_norm_workspace_bytes(T, K), f"rms_norm_workspace_bytes({T}, {K})")
    pd, ph, pw, pr, ps, px, pdw, pws = _pointers(
        (dy, "dy", (T, K), _H), (h, "h", (T, K), _H), weight_spec, (rstd, "rstd", (T,), _F),
        _optional(d_sum, "d_sum", (T, K), _H), (dx, "dx", (T, K), _H), _optional(d_weight, "d_weight", (K,), _F),
        ws_spec)
    _check(lib().moegg_rms_norm_backward(pd, ph, pw, weight_kind, pr, ps, px, pdw, T, K, pws, n,
                                         _stream_for(dy, stream)), "moegg_rms_norm_backward")


@functools.lru_cache(maxsize=4096)
def balance_loss_workspace_bytes(T: int, E: int, S: int = 1) -> int:
    return int(lib().moegg_balance_loss_workspace_bytes(T, E, S))


def balance_loss_workspace(T: int, E: int, S: int = 1, device="cuda") -> torch.Tensor:
    return _workspace_of(balance_loss_workspace_bytes(T, E, S), device)


def balance_loss(logits, ids, loss, counts, ws, *, probs=None, z_loss=None, seq_offsets=None,
                 score: int = SCORE_SOFTMAX, stream=None):
    """The router's balance loss [S] of every sequence from logits [T, E] and the ids [T, k] that route chose, with its
    counts int32 [S, E], mean probabilities probs fp32 [S, E] and z_loss fp32 [S] (see moegg.h).  seq_offsets int32
    [S + 1]: the sequences' bounds; None: all tokens are one.  ws: balance_loss_workspace(T, E, S), or of more."""
    T, E = _matrix(logits, "logits", (_F, _H))
    k = _matrix(ids, "ids", (_I,))[1]
    S = _matrix(counts, "counts", (_I,))[0]
    kind = logits.dtype
    n, ws_spec = _ws_spec(ws, balance_loss_workspace_bytes(T, E, S), f"balance_loss_workspace_bytes({T}, {E}, {S})")
    if seq_offsets is None and S != 1:
        raise ValueError(f"seq_offsets: int32 [{S + 1}] expected for counts of {S} sequences")
    l, i, o, pl, pz, pc, pp, pw = _pointers(
        (logits, "logits", (T, E), kind), (ids, "ids", (T, k), _I), _optional(seq_offsets, "seq_offsets", (S + 1,), _I),
        (loss, "loss", (S,), _F), _optional(z_loss, "z_loss", (S,), _F), (counts, "counts", (S, E), _I),
        _optional(probs, "probs", (S, E), _F), ws_spec)
    _check(lib().moegg_balance_loss(l, LOGITS_BF16 if kind is _H else LOGITS_FP32, i, o, pl, pz, pc, pp, T, E, k, S,
                                    score, pw, n, _stream_for(logits, stream)), "moegg_balance_loss")


def balance_loss_backward(logits, counts, d_loss, d_logits, *, k: int, d_z_loss=None, seq_offsets=None,
                          score: int = SCORE_SOFTMAX, before=None, stream=None):
    """d_logits [T, E] (logits' type) from d_loss [S] and d_z_loss [S], added to `before` [T, E], which may be d_logits
    (see moegg.h); counts as balance_loss wrote them, k the experts of a token."""
    T, E = _matrix(logits, "logits", (_F, _H))
    S = _matrix(counts, "counts", (_I,))[0]
    kind = logits.dtype
    if seq_offsets is None and S != 1:
        raise ValueError(f"seq_offsets: int32 [{S + 1}] expected for counts of {S} sequences")
    l, c, o, dl, dz, b, d = _pointers(
        (logits, "logits", (T, E), kind), (counts, "counts", (S, E), _I),
        _optional(seq_offsets, "seq_offsets", (S + 1,), _I), (d_loss, "d_loss", (S,), _F),
        _optional(d_z_loss, "d_z_loss", (S,), _F), _optional(before, "before", (T, E), kind),
        (d_logits, "d_logits", (T, E), kind))
    _check(lib().moegg_balance_loss_backward(l, LOGITS_BF16 if kind is _H else LOGITS_FP32, c, o, dl, dz, b, d, T, E, k,
                                             S, score, _stream_for(logits, stream)), "moegg_balance_loss_backward")


@functools.lru_cache(maxsize=4096)
def lora_workspace_bytes(T: int, K: int, R: int) -> int:
    return int(lib().moegg_lora_workspace_bytes(T, K, R))


def lora_workspace(T: int, K: int, R: int, device="cuda") -> torch.Tensor:
    return _workspace_of(lora_workspace_bytes(T, K, R), device)


def lora(X, A, B, adapter, Y, out, ws, *, scale=None, stream=None):
    """out[t] = Y[t] + scale[a] * (X[t] A_a^T) B_a^T with a = adapter[t], or Y[t] where that is no adapter (see
    moegg.h).  X bf16 [T, K], Y and out bf16 [T, N] (out may be Y), A bf16 [L, R, K], B bf16 [L, N, R], adapter int32 [T], scale
    fp32 [L].  ws: lora_workspace(T, K, R), or of more rows."""
    T, K = _matrix(X, "X", (_H,))
    N = _matrix(Y, "Y", (_H,))[1]
    if not isinstance(A, torch.Tensor) or A.dim() != 3:
        _need(A, "A", (None, None, K), (_H,))
    L, R = A.shape[0], A.shape[1]
    n, ws_spec = _ws_spec(ws, lora_workspace_bytes(T, K, R), f"lora_workspace_bytes({T}, {K}, {R})")
    px, pa, pb, ps, pi, py, po, pw = _pointers(
        (X, "X", (T, K), _H), (A, "A", (L, R, K), _H), (B, "B", (L, N, R), _H), _optional(scale, "scale", (L,), _F),
        (adapter, "adapter", (T,), _I), (Y, "Y", (T, N), _H), (out, "out", (T, N), _H), ws_spec)
    _check(lib().moegg_lora(px, pa, pb, ps, pi, py, po, T, K, N, R, L, pw, n, _stream_for(X, stream)), "moegg_lora")


def stats_read(ws: torch.Tensor, stream=None) -> Stats:
    s = _Stats()
    _check(lib().moegg_stats_read(_p(ws), ctypes.byref(s), _stream(stream)), "moegg_stats_read")
    return Stats(s.U, s.P_exec, s.tiles, s.active, s.sum_sq, s.capacity_rows,
                 {q: int(s.P_at[i]) for i, q in enumerate(Q_VALUES)}, s.block_m, s.error_flags)


def tile_list_read(ws: torch.Tensor, cap_tiles: int, stream=None) -> List[Tuple[int, int, int, int]]:
    buf = (_Tile * max(1, cap_tiles))()
    n = _I64(0)
    _check(lib().moegg_tile_list_read(_p(ws), buf, cap_tiles, ctypes.byref(n), _stream(stream)),
           "moegg_tile_list_read")
    return [(buf[i].expert, buf[i].tile, buf[i].row_start, buf[i].rows_valid) for i in range(min(n.value, cap_tiles))]
