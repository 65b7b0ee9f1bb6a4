"""Pins of oracle/xattn.py: finite differences, closed forms and the bucket's definition."""
import math

import numpy as np
import pytest

from oracle.xattn import (bucket, bucket_map, head_backward, head_forward, qknorm_backward,
                          qknorm_forward, visible_keys)


def difference(f, x, direction, h=1e-6):
    return (f(x + h * direction) - f(x - h * direction)) / (2 * h)


def test_attention_gradients_are_differences():
    rng = np.random.default_rng(0)
    q, k, v, do = (rng.standard_normal(s) for s in ((5, 8), (7, 8), (7, 8), (5, 8)))
    table = rng.standard_normal(8)
    at = bucket_map(5, 7, 2, 8, 6, True)
    see = visible_keys(5, 7, 6, 2, True)

    def loss(q=q, k=k, v=v, table=table):
        return float((head_forward(q, k, v, 0.3, table[at], see)[0] * do).sum())

    _, _, P = head_forward(q, k, v, 0.3, table[at], see)
    dq, dk, dv, dS = head_backward(q, k, v, P, do, 0.3)
    db = np.bincount(at.ravel(), dS.ravel(), 8)
    for name, x, g in (("q", q, dq), ("k", k, dk), ("v", v, dv), ("table", table, db)):
        d = rng.standard_normal(x.shape)
        want = difference(lambda z, name=name: loss(**{name: z}), x, d)
        assert abs((g * d).sum() - want) < 1e-7 * (1 + abs(want)), name
    assert not dk[6].any() and not dv[6].any()      # behind the sequence's keys


def test_queries_without_keys_give_nothing():
    q, k = np.ones((3, 4)), np.ones((5, 4))
    o, lse, P = head_forward(q, k, k, 1.0, None, np.zeros((3, 5), bool))
    assert not o.any() and np.isneginf(lse).all() and not P.any()
    o, lse, _ = head_forward(q, k[:0], k[:0], 1.0)
    assert not o.any() and np.isneginf(lse).all()


def test_equal_scores_average():
    v = np.arange(12.0).reshape(4, 3)
    o, lse, _ = head_forward(np.zeros((2, 3)), np.zeros((4, 3)), v, 1.0)
    assert np.allclose(o, v.mean(axis=0)) and np.allclose(lse, math.log(4))


@pytest.mark.parametrize("buckets,far,both", [(32, 128, True), (32, 128, False), (16, 64, True),
                                              (8, 5, False), (4, 100, True), (64, 250, False),
                                              (2, 2, False)])
def test_buckets_are_the_definition(buckets, far, both):
    N = buckets // 2 if both else buckets
    E = N // 2
    for n in range(-2 * far - 3, 2 * far + 4):
        a = abs(n) if both else max(-n, 0)
        got = bucket(n, buckets, far, both) - (N if both and n > 0 else 0)
        if a < E:
            assert got == a
            continue
        x = (N - E) * math.log(a / E) / math.log(far / E)
        if abs(x - round(x)) > 1e-9:           # (on a border the logarithms may round down)
            assert got == min(N - 1, E + math.floor(x)), n
        else:
            assert got == min(N - 1, E + round(x)), n
    # where the border is a whole number: 8 * 16^(2/8) = 16 begins a bucket
    assert bucket(-16, 32, 128, True) == bucket(-15, 32, 128, True) + 1


@pytest.mark.parametrize("interleaved", [False, True])
def test_qknorm_gradients_are_differences(interleaved):
    rng = np.random.default_rng(1)
    x, dy, w = rng.standard_normal((3, 2, 8)), rng.standard_normal((3, 2, 8)), rng.standard_normal(8)
    a = rng.uniform(0, 6, (3, 3))
    cos, sin = np.cos(a), np.sin(a)

    def loss(x=x, w=w):
        return float((qknorm_forward(x, w, cos, sin, 1e-3, interleaved) * dy).sum())

    dx, dw = qknorm_backward(x, w, dy, cos, sin, 1e-3, interleaved)
    for name, z, g in (("x", x, dx), ("w", w, dw)):
        d = rng.standard_normal(z.shape)
        want = difference(lambda t, name=name: loss(**{name: t}), z, d)
        assert abs((g * d).sum() - want) < 1e-7 * (1 + abs(want)), name


def test_rotation_keeps_lengths_and_relative_positions():
    """|y| is |w x r| and the product of a query at p and a key at s depends on p - s."""
    rng = np.random.default_rng(2)
    x, z = rng.standard_normal((2, 1, 1, 6))
    freq = np.array([1.0, 0.1, 0.01])

    def turned(x, p):
        return qknorm_forward(x, np.ones(6), np.cos(p * freq)[None], np.sin(p * freq)[None], 1e-9, False)

    assert np.isclose(np.linalg.norm(turned(x, 5)), math.sqrt(6))
    assert np.isclose((turned(x, 5) * turned(z, 3)).sum(), (turned(x, 9) * turned(z, 7)).sum())
