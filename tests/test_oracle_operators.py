"""Pins of the oracle's gated feed-forward block and linear-head cross entropy
(oracle/glu.py, oracle/head.py): closed forms, finite differences, shard sums."""
import numpy as np
import pytest

from oracle.glu import act_and_grad, glu_backward, glu_output, glu_projections
from oracle.head import ce_backward, ce_forward


def _glu(M=5, H=4, F=6, bias=True, seed=0):
    r = np.random.default_rng(seed)
    w = {"w1": r.normal(size=(2 * F, H)), "w2": r.normal(size=(H, F))}
    if bias:
        w |= {"b1": r.normal(size=2 * F), "b2": r.normal(size=H)}
    return r.normal(size=(M, H)), r.normal(size=(M, H)), w


def _run(x, w, act, resid=None):
    return glu_output(*glu_projections(x, w), w, act, resid)


def test_activations_at_known_points():
    f, d = act_and_grad(np.array([0.0, 1.0, -1.0]), "silu")
    s = 1 / (1 + np.exp(-1.0))
    np.testing.assert_allclose(f, [0.0, s, -(1 - s)], rtol=1e-15)
    np.testing.assert_allclose(d, [0.5, s * (2 - s), (1 - s) * (1 - s)], rtol=1e-14)
    f, d = act_and_grad(np.array([0.0, 1.0]), "gelu")
    np.testing.assert_allclose(f, [0.0, 0.841344746068543], rtol=1e-12)
    np.testing.assert_allclose(d[0], 0.5, rtol=1e-15)


def test_constant_gate_makes_a_linear_map():
    """Wg = 0, bg = c: y = act(c) x Wu^T W2^T."""
    x, _, w = _glu(bias=False)
    F = w["w2"].shape[1]
    w["w1"][:F] = 0.0
    w["b1"] = np.r_[np.full(F, 0.7), np.zeros(F)]
    for act in ("silu", "gelu"):
        c = act_and_grad(np.array(0.7), act)[0]
        np.testing.assert_allclose(_run(x, w, act), c * x @ w["w1"][F:].T @ w["w2"].T, rtol=1e-12)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_glu_gradients_are_finite_differences(act):
    x, g, w = _glu()
    resid = np.random.default_rng(3).normal(size=x.shape)
    dx, grads = glu_backward(g, x, *glu_projections(x, w), w, act)
    eps = 1e-6

    def loss(xx, ww):
        return (_run(xx, ww, act, resid) * g).sum()

    for name, v, got in [("x", x, dx)] + [(k, w[k], grads[k]) for k in w]:
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[i] = eps
            up = (x + d, w) if name == "x" else (x, {**w, name: v + d})
            dn = (x - d, w) if name == "x" else (x, {**w, name: v - d})
            num[i] = (loss(*up) - loss(*dn)) / (2 * eps)
        np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("shards", [2, 3])
def test_shard_partials_sum_to_the_block(shards):
    """Shard k: rows [k F/w, ...) of Wg and Wu, the same columns of W2."""
    x, _, w = _glu(bias=False)
    F, total = w["w2"].shape[1], 0.0
    for k in range(shards):
        part = slice(k * F // shards, (k + 1) * F // shards)
        total = total + _run(x, {"w1": np.r_[w["w1"][:F][part], w["w1"][F:][part]],
                                 "w2": w["w2"][:, part]}, "silu")
    np.testing.assert_allclose(total, _run(x, w, "silu"), rtol=1e-12)


def test_ce_closed_forms():
    x, w = np.zeros((2, 3)), np.random.default_rng(0).normal(size=(7, 3))
    loss, lse, _ = ce_forward(x, w, np.array([0, 6]))
    np.testing.assert_allclose(loss, np.log(7.0), rtol=1e-15)
    dx, dw, g = ce_backward(x, w, np.array([0, 6]), np.ones(2))
    np.testing.assert_allclose(g.sum(axis=1), 0.0, atol=1e-15)
    np.testing.assert_allclose(dx[0], w.mean(axis=0) - w[0], rtol=1e-12)
    assert not dw.any()
    # two classes: loss = log(1 + e^(l1 - l0))
    loss, _, _ = ce_forward(np.array([[1.0]]), np.array([[0.3], [1.1]]), np.array([0]))
    np.testing.assert_allclose(loss, np.log1p(np.exp(0.8)), rtol=1e-14)


def test_ce_gradients_are_finite_differences_and_ignored_rows_have_none():
    r = np.random.default_rng(1)
    x, w, t = r.normal(size=(4, 3)), r.normal(size=(6, 3)), np.array([2, -100, 5, 2])
    d = r.normal(size=4)
    dx, dw, _ = ce_backward(x, w, t, d)
    eps = 1e-6
    for v, got, at in ((x, dx, 0), (w, dw, 1)):
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            e = np.zeros_like(v)
            e[i] = eps
            up, dn = ([x, w], [x, w])
            up[at], dn[at] = v + e, v - e
            num[i] = ((ce_forward(*up, t)[0] - ce_forward(*dn, t)[0]) * d).sum() / (2 * eps)
        np.testing.assert_allclose(got, num, rtol=1e-6, atol=1e-8)
    assert ce_forward(x, w, t)[0][1] == 0.0 and not dx[1].any()
    # an extreme logit neither overflows nor loses the others
    loss, lse, _ = ce_forward(np.array([[1e4]]), np.array([[1.0], [0.0]]), np.array([1]))
    assert loss[0] == pytest.approx(1e4)
