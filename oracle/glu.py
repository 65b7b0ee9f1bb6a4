"""Gated feed-forward block, float64 numpy (oracle; test infrastructure only).

Not on the Oases pages; the textbook definition, in the layout of the C ABI:
  a = x Wg^T + bg, b = x Wu^T + bu with w1 = [Wg; Wu] [2F, H], b1 = [bg, bu],
  h = act(a) * b, y = h W2^T + b2 (+ resid).
act: SiLU a / (1 + e^-a), or the exact GeLU of ``oracle.ops``.
Pinned by finite differences, closed forms (W2 = identity, constant gates) and
the sum of shard partials in tests/test_oracle_operators.py.
"""
from __future__ import annotations

import numpy as np
from scipy.special import expit

from .ops import gelu, gelu_grad


def act_and_grad(a: np.ndarray, act: str):
    if act == "silu":
        s = expit(a)
        return a * s, s * (1.0 + a * (1.0 - s))
    assert act == "gelu", act
    return gelu(a), gelu_grad(a)


def glu_projections(x, w):
    """(a, b) [M, F]."""
    p = x @ w["w1"].T
    if w.get("b1") is not None:
        p = p + w["b1"]
    F = w["w2"].shape[1]
    return p[:, :F], p[:, F:]


def glu_output(a, b, w, act, resid=None):
    """y from the projections."""
    y = (act_and_grad(a, act)[0] * b) @ w["w2"].T
    if w.get("b2") is not None:
        y = y + w["b2"]
    return y if resid is None else y + resid


def glu_backward(dy, x, a, b, w, act):
    """(dx, {w1, b1, w2, b2}) at the projections (a, b):
    dh = dy W2; da = dh b act'(a); db = dh act(a); dx = [da db] W1;
    dW1 = [da db]^T x; db1 = colsum [da db]; dW2 = dy^T h; db2 = colsum dy."""
    f, df = act_and_grad(a, act)
    dh = dy @ w["w2"]
    dp = np.concatenate([dh * b * df, dh * f], axis=1)
    return dp @ w["w1"], {"w1": dp.T @ x, "b1": dp.sum(axis=0), "w2": dy.T @ (f * b),
                          "b2": dy.sum(axis=0)}
