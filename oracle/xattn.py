"""Attention over keys of another length with a relative position bias, and the norms per
head with the position rotation, float64 numpy (oracle; test infrastructure only).

Not on the Oases pages; the textbook definitions, in the layout of the C ABI
(oases_attn.h, oases_qknorm.h).  Pinned by finite differences and closed forms in
tests/test_oracle_attn.py.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np


# ---- buckets of relative positions -------------------------------------------------
def bucket(n: int, buckets: int, max_distance: int, bidirectional: bool) -> int:
    """The bucket of relative position n (the key's minus the query's): whole arithmetic
    decides E + floor((N - E) log(a / E) / log(max_distance / E))."""
    N = buckets // 2 if bidirectional else buckets
    upper = N if bidirectional and n > 0 else 0
    a = abs(n) if bidirectional else max(-n, 0)
    E = N // 2
    if a < E:
        return upper + a
    ratio, top = Fraction(a, E) ** (N - E), Fraction(max_distance, E)
    u = 0
    while u < N - 1 - E and top ** (u + 1) <= ratio:
        u += 1
    return upper + E + u


def bucket_map(q_len, k_len, start, buckets, max_distance, bidirectional):
    """[q_len, k_len] buckets of j - (start + i)."""
    n = np.arange(k_len)[None, :] - (start + np.arange(q_len))[:, None]
    low, high = (int(n.min()), int(n.max())) if n.size else (0, 0)
    known = np.array([bucket(x, buckets, max_distance, bidirectional) for x in range(low, high + 1)])
    return known[n - low]


# ---- attention of one sequence and head ------------------------------------------------
def head_forward(q, k, v, scale, bias=None, visible=None):
    """(o, lse, P) of q [Sq, D] over k, v [Sk, D]; bias [Sq, Sk] added to the scores,
    visible [Sq, Sk] truth values.  A query that sees nothing: o = 0, lse = -inf."""
    s = scale * (q @ k.T)
    if bias is not None:
        s = s + bias
    if visible is not None:
        s = np.where(visible, s, -np.inf)
    top = s.max(axis=1, initial=-np.inf)
    top = np.where(np.isneginf(top), 0.0, top)
    e = np.exp(s - top[:, None])
    total = e.sum(axis=1)
    P = e / np.where(total > 0, total, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        return P @ v, top + np.log(total), P


def head_backward(q, k, v, P, do, scale):
    """(dq, dk, dv, dS) from the weights P."""
    dP = do @ v.T
    dS = P * (dP - (P * dP).sum(axis=1, keepdims=True))
    return scale * (dS @ k), scale * (dS.T @ q), P.T @ do, dS


def visible_keys(q_len, k_len, length, start, causal):
    j = np.arange(k_len)[None, :]
    see = np.broadcast_to(j < length, (q_len, k_len))
    return see & (j <= start + np.arange(q_len)[:, None]) if causal else see


# ---- norms per head and the rotation -----------------------------------------------------
def _rotation(x, cos, sin, interleaved, sign):
    """The rotation of x [tokens, heads, D] by cos, sin [tokens, rot / 2] (transposed
    with sign -1)."""
    R = 2 * cos.shape[1]
    y = x.copy()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    c, s = cos[:, None], sign * sin[:, None]
    y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
    return y


def qknorm_forward(x, w, cos, sin, eps, interleaved):
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    return _rotation(x * r * w, cos, sin, interleaved, 1.0)


def qknorm_backward(x, w, dy, cos, sin, eps, interleaved):
    """(dx, dw)."""
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    g = _rotation(dy, cos, sin, interleaved, -1.0)
    m = (g * w * x * r).mean(axis=-1, keepdims=True)
    return r * (g * w - x * r * m), (g * x * r).sum(axis=(0, 1))
