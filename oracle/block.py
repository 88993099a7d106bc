"""The operators around the MoE layer, in fp64 from their definitions (test infrastructure only).

- rms_norm / rms_norm_backward: values before they are stored in a format.
- balance_loss / balance_loss_backward: sequence by sequence.
- lora: row by row.

Everything is numpy.
"""
from __future__ import annotations

from typing import List, Optional, Tuple

import numpy as np

from .layer import FLT_MAX, scores


# ------------------------------------------------------------------ norm

def rms_norm(h, weight, eps: float):
    """(h rstd weight, rstd)."""
    h = np.asarray(h, dtype=np.float64)
    rstd = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h * rstd[:, None] * np.asarray(weight, dtype=np.float64), rstd


def rms_norm_backward(dy, h, weight, rstd, d_sum=None):
    """(dx, d_weight) for the rstd given."""
    xhat = h * rstd[:, None]
    g = dy * weight
    dx = rstd[:, None] * (g - xhat * (g * xhat).mean(axis=1, keepdims=True))
    return dx + (0.0 if d_sum is None else d_sum), (dy * xhat).sum(axis=0)


# ------------------------------------------------------------------ balance loss

def bounds(offsets, T: int) -> List[Tuple[int, int]]:
    """[start, end) of every sequence, within [0, T]."""
    if offsets is None:
        return [(0, T)]
    o = [min(max(int(v), 0), T) for v in offsets]
    return [(a, max(a, b)) for a, b in zip(o[:-1], o[1:])]


def clean(logits):
    l = np.asarray(logits, dtype=np.float64)
    return np.where(np.isnan(l), -np.inf, np.minimum(l, FLT_MAX))


def log_sum_exp(logits):
    """[T]; 0 for a token without experts."""
    l = clean(logits)
    m = l.max(axis=1)
    there = m > -np.inf
    safe = np.where(there, m, 0.0)
    with np.errstate(divide="ignore", over="ignore"):
        s = np.exp(l - safe[:, None]).sum(axis=1)
        return np.where(there, safe + np.log(np.where(there, s, 1.0)), 0.0)


def probabilities(logits, score: str):
    """p [T, E]: softmax, or sigmoids over their sum (through their logarithms, so that none is lost)."""
    if score == "softmax":
        return scores(logits, score)
    ln = -np.logaddexp(0.0, -clean(logits))
    m = ln.max(axis=1, keepdims=True)
    e = np.exp(ln - np.where(m > -np.inf, m, 0.0))
    z = e.sum(axis=1, keepdims=True)
    return e / np.where(z > 0, z, 1.0)


def balance_loss(logits, ids, offsets=None, score: str = "softmax"):
    """loss [S], z [S], counts [S, E], probs [S, E]."""
    T, E = np.shape(logits)
    k = np.shape(ids)[1]
    b = bounds(offsets, T)
    loss, z = np.zeros(len(b)), np.zeros(len(b))
    counts, probs = np.zeros((len(b), E), dtype=np.int64), np.zeros((len(b), E))
    p, lse = probabilities(logits, score), log_sum_exp(logits)
    for s, (start, end) in enumerate(b):
        n = end - start
        if n == 0:
            continue
        for e in np.asarray(ids)[start:end].reshape(-1):
            if 0 <= e < E:
                counts[s, e] += 1
        probs[s] = p[start:end].mean(axis=0)
        loss[s] = E / (k * n) * (counts[s] * probs[s]).sum()
        z[s] = (lse[start:end] ** 2).mean()
    return loss, z, counts, probs


def balance_loss_backward(logits, counts, d_loss, k: int, d_z=None, offsets=None, score: str = "softmax", before=None):
    """d_logits [T, E], by the Jacobian of each token's probabilities."""
    T, E = np.shape(logits)
    d = np.zeros((T, E)) if before is None else np.array(before, dtype=np.float64)
    l, p, lse = clean(logits), probabilities(logits, score), log_sum_exp(logits)
    with np.errstate(over="ignore"):
        rest = 1.0 / (1.0 + np.exp(l))                       # 1 - sigmoid
    for s, (start, end) in enumerate(bounds(offsets, T)):
        n = end - start
        for t in range(start, end):
            g = d_loss[s] * E / (k * n) * counts[s] / n
            dp = p[t] * (g - (p[t] * g).sum())
            d[t] += dp if score == "softmax" else dp * rest[t]
            if d_z is not None:
                d[t] += d_z[s] * 2 * lse[t] / n * p[t]
    return d


# ------------------------------------------------------------------ adapters

def lora(X, A, B, adapter, Y, scale: Optional[np.ndarray] = None):
    """out [T, N], row by row."""
    out = np.array(Y, dtype=np.float64)
    for t, a in enumerate(adapter):
        if 0 <= a < len(A):
            out[t] += (1.0 if scale is None else scale[a]) * (B[a] @ (A[a] @ X[t]))
    return out
