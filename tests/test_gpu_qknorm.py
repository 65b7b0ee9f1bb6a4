"""Norms of queries and keys per head with the position rotation (oases_qknorm.h) on the
GPU, against the float64 definition (oracle/xattn.py), element by element.

Bounds.  u = 2^-8 (bf16) or 2^-24 (fp32) is half a step of the storage type; e = 2^-24
that of fp32.  A sum over D terms is off by at most D 2^-23 of the terms' sizes, so
with G = (D + 12) 2^-23 for the statistics and the dozen roundings of a value:
  y    G (|a c| + |b s|) + u |y|
  dx   G r (|g w| + |x r| mean |g w x r|) twice over (g and the mean) + u |dx|
  dw   sum (G + n 2^-23) |g x r| + u |dw|
with a factor 1.05 for the products of errors; nothing is fitted.
"""
import numpy as np
import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from oracle.xattn import _rotation, qknorm_backward, qknorm_forward
from tensor_model_transformer_tp_gb300 import functional as F

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
SLACK = 1.05


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def f64(t):
    return t.detach().double().cpu().numpy()


def inside(got, want, bound, what):
    got = f64(got)
    bad = ~(np.abs(got - want) <= SLACK * bound + 1e-30)
    assert not bad.any(), "%s: %d of %d off, first at %s (%r, want %r)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[tuple(np.argwhere(bad)[0])],
        want[tuple(np.argwhere(bad)[0])])


def inputs(dtype, B, S, H, G, D, rot, P, seed=0):
    gen = torch.Generator().manual_seed(seed + B + 3 * S + 5 * H + 7 * D + rot)

    def rnd(*shape, std=1.0, mean=0.0):
        return (torch.randn(*shape, generator=gen) * std + mean).to(T[dtype]).cuda()

    qkv = rnd(B, S, H + 2 * G, D)
    angle = torch.arange(P, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))
    return {"q": qkv[:, :, :H], "k": qkv[:, :, H:H + G], "dq": rnd(B, S, H, D),
            "dk": rnd(B, S, G, D), "wq": rnd(D, std=0.2, mean=1.0), "wk": rnd(D, std=0.2, mean=1.0),
            "cos": angle.cos().float().cuda(), "sin": angle.sin().float().cuda(),
            "positions": torch.randint(P, (B, S), generator=gen).cuda()}


def check(dtype, x, w, dy, cos, sin, eps, il, y, dx, dw, what):
    """x, dy [B, S, heads, D]; cos, sin [B S, rot / 2]."""
    u, D = U[dtype], x.shape[-1]
    x, dy = (f64(t).reshape(-1, t.shape[2], D) for t in (x, dy))
    w = np.ones(D) if w is None else f64(w)
    G = (D + 12) * 2.0 ** -23
    r = 1.0 / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps)
    want = qknorm_forward(x, w, cos, sin, eps, il)

    def turned(v):      # |a c| + |b s|
        return np.abs(_rotation(np.abs(v), np.abs(cos), np.abs(sin), il, 1.0)) + \
            np.abs(_rotation(np.abs(v), np.abs(cos), np.abs(sin), il, -1.0))

    inside(y.reshape(want.shape), want, G * turned(x * r * w) + u * np.abs(want), what)
    if dx is None:
        return
    want, want_w = qknorm_backward(x, w, dy, cos, sin, eps, il)
    gs = turned(dy)
    inside(dx.reshape(want.shape), want, 2 * G * r * (
        gs * np.abs(w) + np.abs(x * r) * (gs * np.abs(w * x * r)).mean(axis=-1, keepdims=True)) +
        u * np.abs(want), "d" + what)
    if dw is not None:
        n = x.shape[0] * x.shape[1]
        inside(dw, want_w, (G + n * 2.0 ** -23) * (gs * np.abs(x * r)).sum(axis=(0, 1)) +
               u * np.abs(want_w), "dw of " + what)


# (batch, tokens, heads, key heads, head size, values turned)
SHAPES = [(1, 1, 1, 1, 8, 8), (64, 1, 32, 8, 128, 128), (3, 17, 6, 2, 80, 32), (2, 33, 5, 5, 64, 64),
          (1, 130, 3, 1, 40, 40), (2, 9, 2, 1, 256, 64), (1, 77, 1, 4, 16, 10), (2, 50, 20, 20, 128, 128),
          (1, 19, 7, 3, 96, 24), (4, 300, 9, 2, 72, 2), (1, 5, 2, 2, 24, 0)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(dtype, interleaved, shape):
    B, S, H, G, D, rot = shape
    P = 700
    s = inputs(dtype, *shape, P)
    for positions in (None, s["positions"], s["positions"][0].contiguous()):
        at = torch.arange(S).expand(B, S) if positions is None else positions.cpu().expand(B, S)
        cos, sin = (f64(s[n])[at.reshape(-1).numpy()] for n in ("cos", "sin"))
        opt = dict(positions=positions, q_weight=s["wq"], k_weight=s["wk"], eps=1e-5,
                   interleaved=interleaved)
        q, k = F.qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], **opt)
        dq, dk, dwq, dwk = F.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"],
                                              **opt)
        check(dtype, s["q"], s["wq"], s["dq"], cos, sin, 1e-5, interleaved, q, dq, dwq, "q")
        check(dtype, s["k"], s["wk"], s["dk"], cos, sin, 1e-5, interleaved, k, dk, dwk, "k")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_parts_left_out(dtype):
    """No weights, no keys, no rotation: the same values as with weights of 1, keys
    beside and angles of 0."""
    s = inputs(dtype, 2, 30, 4, 2, 64, 64, 50)
    one = torch.ones(64, dtype=T[dtype], device="cuda")
    zero = torch.zeros_like(s["sin"])
    q, k = F.qk_norm_rope_fwd(s["q"], s["k"], zero + 1.0, zero, q_weight=one, k_weight=one)
    q2, none = F.qk_norm_rope_fwd(s["q"], None, None, None)
    assert none is None and torch.equal(q, q2)
    assert torch.equal(k, F.qk_norm_rope_fwd(s["k"], None, None, None, q_weight=one)[0])
    dq, dk, dwq, dwk = F.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"],
                                          q_weight=one)
    assert dwk is None and dwq is not None
    dq2, dk2, dwq2, dwk2 = F.qk_norm_rope_bwd(s["q"], None, s["dq"], None, s["cos"], s["sin"],
                                              q_weight=one)
    assert torch.equal(dq, dq2) and dk2 is None and dwk2 is None
    assert (dwq.double() - dwq2.double()).abs().max() <= 2.0 ** -6 * dwq.double().abs().max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (24, False), (40, False)])
def test_in_place_and_accumulated(dtype, rot, interleaved):
    s = inputs(dtype, 2, 65, 5, 3, 64, rot, 70)
    opt = dict(q_weight=s["wq"], k_weight=s["wk"], interleaved=interleaved)
    q, k = F.qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], **opt)
    back = F.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"], **opt)
    grads = [torch.full((64,), 2.0, device="cuda") for _ in range(2)]
    zeros = [torch.zeros(64, device="cuda") for _ in range(2)]
    dq, dk = s["dq"].clone(), s["dk"].clone()
    got = F.qk_norm_rope_bwd(s["q"], s["k"], dq, dk, s["cos"], s["sin"], out=(dq, dk), grads=grads,
                             **opt)
    assert got[0] is dq and got[2] is grads[0]
    F.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"], grads=zeros, **opt)
    for a, b, c in zip(back[2:], grads, zeros):
        assert torch.equal(c + 2.0, b) and torch.equal(c.to(T[dtype]), a)
    assert torch.equal(dq, back[0]) and torch.equal(dk, back[1])
    x, y = s["q"].clone(), s["k"].clone()
    F.qk_norm_rope_fwd(x, y, s["cos"], s["sin"], out=(x, y), **opt)
    assert torch.equal(x, q) and torch.equal(y, k)


def test_positions_outside_the_tables_are_nan_in_their_token_alone():
    s = inputs("bf16", 1, 6, 2, 1, 64, 32, 10)
    at = torch.tensor([[0, 9, 10, -1, 3, 1 << 40]], device="cuda")
    q, k = F.qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], positions=at)
    bad = torch.tensor([False, False, True, True, False, True], device="cuda")
    for y in (q, k):
        assert torch.isnan(y[0, bad][..., :32]).all() and torch.isfinite(y[0, bad][..., 32:]).all()
        assert torch.isfinite(y[0, ~bad]).all()


def test_captured_and_empty():
    s = inputs("bf16", 3, 40, 4, 2, 128, 128, 64)
    opt = dict(positions=s["positions"], q_weight=s["wq"], k_weight=s["wk"])
    args = (s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"])
    want = F.qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], **opt) + F.qk_norm_rope_bwd(*args, **opt)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = F.qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], **opt) + F.qk_norm_rope_bwd(*args, **opt)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    e = inputs("f32", 0, 7, 2, 1, 64, 64, 10)
    q, k = F.qk_norm_rope_fwd(e["q"], e["k"], e["cos"], e["sin"], q_weight=e["wq"])
    _, _, dwq, _ = F.qk_norm_rope_bwd(e["q"], e["k"], e["dq"], e["dk"], e["cos"], e["sin"], q_weight=e["wq"])
    assert q.shape == e["q"].shape and not dwq.any()
