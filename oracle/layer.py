"""The operators around the grouped GEMMs, in fp64 from their definitions (test infrastructure only).

- route / route_backward: router logits -> expert ids, weights, counts and rows; the gradient of the logits.
- dispatch / combine / combine_backward: values of the rows, before they are stored in an operand format.
- swiglu / swiglu_backward: on the interleaved gate/up columns.
- row_scales, token_groups: the groups that share a scale, and amax / 448.

Everything is numpy, token by token or group by group.
"""
from __future__ import annotations

from typing import List, Optional, Sequence, Tuple

import numpy as np

from .mlp import split_gate_up

FLT_MAX = float(np.finfo(np.float32).max)
E4M3_MAX = 448.0


# ------------------------------------------------------------------ routing

def scores(logits: np.ndarray, score: str) -> np.ndarray:
    """fp64 scores [T, E]; NaN logits count as -inf, +inf as the largest fp32 number."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, FLT_MAX))
    with np.errstate(over="ignore", invalid="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-l))
        top = l.max(axis=1, keepdims=True)
        e = np.where(l > -np.inf, np.exp(l - np.where(top > -np.inf, top, 0.0)), 0.0)
        z = e.sum(axis=1, keepdims=True)
        return e / np.where(z > 0, z, 1.0)


def route(logits, k: int, score: str = "softmax", bias=None, n_groups: int = 1, topk_groups: int = 1,
          group_top: int = 1, renorm: bool = True, scale: float = 1.0):
    """ids int [T, k] (-1: none) and fp64 weights [T, k], one token at a time."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, FLT_MAX))
    s = scores(logits, score)
    T, E = l.shape
    gs = E // n_groups
    b = None if bias is None else np.minimum(np.asarray(bias, dtype=np.float64), FLT_MAX)
    ids = np.full((T, k), -1, dtype=np.int64)
    w = np.zeros((T, k))
    for t in range(T):
        ok = [l[t, e] > -np.inf and (b is None or b[e] > -np.inf) for e in range(E)]
        key = [(l[t, e] if b is None else s[t, e] + b[e]) if ok[e] else -np.inf for e in range(E)]
        kept = range(n_groups)
        if n_groups > 1:
            # a group of single best experts is ordered by their keys, a sum of two by scores (with the bias)
            gk = key if b is not None or group_top == 1 else [s[t, e] if ok[e] else -np.inf for e in range(E)]
            # of the scores that there are; a group without any is below all others
            have = [[x for x in gk[i * gs:(i + 1) * gs] if x > -np.inf] for i in range(n_groups)]
            g = [sum(sorted(x, reverse=True)[:group_top]) if x else -np.inf for x in have]
            kept = sorted(range(n_groups), key=lambda i: (-g[i], i))[:topk_groups]
        cand = [e for e in range(E) if e // gs in kept and ok[e]]
        pick = sorted(cand, key=lambda e: (-key[e], e))[:k]
        ids[t, :len(pick)] = pick
        w[t, :len(pick)] = weights(l[t, pick], s[t, pick], score, renorm, scale)
    return ids, w


def weights(l: np.ndarray, s: np.ndarray, score: str, renorm: bool, scale: float) -> np.ndarray:
    """Weights of one token's chosen experts (logits l, scores s)."""
    if not renorm or len(l) == 0:
        return scale * s
    with np.errstate(over="ignore"):
        # ln of the score, so that far negative logits keep their ratio
        ln = l if score == "softmax" else -np.logaddexp(0.0, -l)
        r = np.exp(ln - ln.max())
    return scale * r / r.sum()


def rows_of(ids: np.ndarray, E: int, rows_total: int, seg_align: int = 1, cap: int = 0) -> Tuple[np.ndarray, np.ndarray]:
    """(m_sizes [E], row_of [T, k]), assignment by assignment in token order."""
    T, k = ids.shape
    m = np.zeros(E, dtype=np.int64)
    rank = np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        for j in range(k):
            if ids[t, j] >= 0:
                rank[t, j] = m[ids[t, j]]
                m[ids[t, j]] += 1
    start = [0]
    for e in range(E):
        start.append(start[-1] + (int(m[e]) + seg_align - 1) // seg_align * seg_align)
    row = np.full((T, k), -1, dtype=np.int64)
    for t in range(T):
        for j in range(k):
            if ids[t, j] < 0:
                continue
            e, r = int(ids[t, j]), int(rank[t, j])
            if cap:
                row[t, j] = e * cap + r if r < cap and e * cap + r < rows_total else -1
            else:
                row[t, j] = start[e] + r if start[e] + r < rows_total else -1
    return m, row


def route_backward(logits, ids: np.ndarray, d_weights, score: str = "softmax", renorm: bool = True,
                   scale: float = 1.0) -> np.ndarray:
    """d_logits fp64 [T, E] by the chain rule through the scores' Jacobian, one token at a time."""
    l = np.asarray(logits, dtype=np.float64)
    s = scores(logits, score)
    dw = np.asarray(d_weights, dtype=np.float64)
    T, E = l.shape
    out = np.zeros((T, E))
    for t in range(T):
        at = [j for j in range(ids.shape[1]) if 0 <= ids[t, j] < E]
        c = ids[t, at]
        ds = np.zeros(E)
        if renorm and score == "softmax":                  # a softmax over the chosen alone: no other logit enters
            z = s[t, c].sum()
            p = s[t, c] / z if z > 0 else s[t, c]
            out[t, c] = scale * (np.diag(p) - np.outer(p, p)) @ dw[t, at]
            continue
        if renorm:
            z = s[t, c].sum()
            if z > 0:
                ds[c] = scale * (dw[t, at] / z - (dw[t, at] * s[t, c]).sum() / z ** 2)
        else:
            ds[c] = scale * dw[t, at]
        if score == "softmax":
            J = np.diag(s[t]) - np.outer(s[t], s[t])
            out[t] = J @ ds
        else:
            out[t] = ds * s[t] * (1 - s[t])
    return out


# ------------------------------------------------------------------ permutation

def assignments(row_of: np.ndarray, rows: int) -> List[Tuple[int, int, int]]:
    """(t, j, row) of every assignment that has a row."""
    T, k = row_of.shape
    return [(t, j, int(row_of[t, j])) for t in range(T) for j in range(k) if 0 <= row_of[t, j] < rows]


def dispatch(x: np.ndarray, row_of: np.ndarray, rows: int) -> dict:
    return {r: np.asarray(x[t], dtype=np.float64) for t, j, r in assignments(row_of, rows)}


def combine(Y: np.ndarray, row_of: np.ndarray, w: Optional[np.ndarray], rows: int) -> Tuple[np.ndarray, np.ndarray]:
    """(out fp64 [T, N], the sums of the terms' magnitudes)."""
    out = np.zeros((row_of.shape[0], Y.shape[1]))
    mag = np.zeros_like(out)
    for t, j, r in assignments(row_of, rows):
        term = Y[r].astype(np.float64) * (1.0 if w is None else float(w[t, j]))
        out[t] += term
        mag[t] += np.abs(term)
    return out, mag


def combine_backward(dout, Y, w, row_of, rows):
    """({row: dY row}, d_weights fp64 [T, k], sums of the dot products' terms' magnitudes)."""
    dY, dw, mag = {}, np.zeros(row_of.shape), np.zeros(row_of.shape)
    for t, j, r in assignments(row_of, rows):
        d = dout[t].astype(np.float64)
        dY[r] = float(w[t, j]) * d
        p = Y[r].astype(np.float64) * d
        dw[t, j], mag[t, j] = p.sum(), np.abs(p).sum()
    return dY, dw, mag


# ------------------------------------------------------------------ SwiGLU

def interleave(g: np.ndarray, u: np.ndarray) -> np.ndarray:
    """[R, I] gate and up -> [R, 2I] in blocks of 16."""
    out = np.empty((g.shape[0], 2 * g.shape[1]))
    col = np.arange(g.shape[1])
    at = 32 * (col // 16) + col % 16
    out[:, at], out[:, at + 16] = g, u
    return out


def sigmoid(x):
    """sigmoid(x), 0 where it is below the smallest normal fp32 number, 2^-126 (x < -87.3), as the calls define it."""
    with np.errstate(over="ignore"):
        s = 1.0 / (1.0 + np.exp(-x))
    return np.where(s < 2.0 ** -126, 0.0, s)


def swiglu(gu: np.ndarray) -> np.ndarray:
    g, u = split_gate_up(np.asarray(gu, dtype=np.float64))
    return g * sigmoid(g) * u


def swiglu_backward(gu: np.ndarray, dh: np.ndarray) -> Tuple[np.ndarray, np.ndarray]:
    """(dGU [R, 2I], h [R, I]) by the derivative of g sigmoid(g) u."""
    g, u = split_gate_up(np.asarray(gu, dtype=np.float64))
    s = sigmoid(g)
    return interleave(dh * u * (s + g * s * sigmoid(-g)), dh * g * s), g * s * u


# ------------------------------------------------------------------ scales

def scale_of(amax: np.ndarray, pow2: bool) -> np.ndarray:
    s = np.asarray(amax, dtype=np.float64) / E4M3_MAX
    s = np.where(s > 0, s, 1.0)
    if pow2:
        m, e = np.frexp(s)
        s = np.exp2(np.maximum(np.where(m == 0.5, e - 1, e), -126))
    return s


def row_scales(v: np.ndarray, pow2: bool = False) -> np.ndarray:
    """[R, K/128] scales of 1x128 groups."""
    return scale_of(np.abs(v.reshape(v.shape[0], -1, 128)).max(axis=2), pow2)


def token_groups(counts: Sequence[int], rows: int) -> List[Tuple[int, int]]:
    """(first row, end) of every token group, in order: up to 128 rows of one expert's segment."""
    out, at = [], 0
    for c in counts:
        end = min(at + max(int(c), 0), rows)
        out += [(r, min(r + 128, end)) for r in range(at, end, 128)]
        at = end
    return out
