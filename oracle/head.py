"""Cross entropy of a linear head, float64 numpy (oracle; test infrastructure only).

Not on the Oases pages; the textbook definition: logits l = x W^T,
lse = log sum exp l, loss = lse - l[target]; rows with target == ignore have
loss 0 and no gradient.  Pinned by closed forms and finite differences in
tests/test_oracle_operators.py.
"""
from __future__ import annotations

import numpy as np


def ce_forward(x, w, target, ignore=-100):
    """(loss, lse, logits)."""
    l = x @ w.T
    top = l.max(axis=1)
    lse = top + np.log(np.exp(l - top[:, None]).sum(axis=1))
    used = target != ignore
    at = np.where(used, target, 0)
    return np.where(used, lse - l[np.arange(len(at)), at], 0.0), lse, l


def ce_backward(x, w, target, dloss, ignore=-100):
    """(dx, dw, g) for the gradient dloss [M] of the losses:
    g = (softmax - onehot) dloss, dx = g W, dW = g^T x."""
    _, lse, l = ce_forward(x, w, target, ignore)
    used = target != ignore
    g = np.exp(l - lse[:, None])
    g[np.arange(len(target))[used], target[used]] -= 1.0
    g = g * np.where(used, dloss, 0.0)[:, None]
    return g @ w, g.T @ x, g
