"""Attention over keys of another length with a relative position bias (oases_attn.h) on
the GPU, against the float64 definition (oracle/xattn.py), element by element.

Bounds.  u = 2^-8 (bf16) or 2^-24 (fp32) is half a step of the storage type relative to
the value; a product over K terms accumulated in fp32 in any order, truncated or
rounded, is off by at most g(K) sum |terms|, g(K) = K 2^-23.  The exponential and the
arithmetic around it are given EW = 2^-18 relative, the score beside its product three
roundings.  So, first order in those:
  s        es = g(D) scale |q||k| + 3 2^-23 (|s| + |bias|)
  P        rP = es + (sum P es) + EW relative; as an operand U more (bf16: u, fp32: 0)
  o        sum P (rP + U) |v| + g(n) sum P |v| + u |o|
  dP       ed = g(D) |do||v|;   delta  et = |do| . (u |o| + error of o) + g(D) |do||o|
  dS       eS = P (rP |dP - delta| + ed + et)
  dq       scale (sum eS |k| + (U + g(n)) sum |dS||k|) + u |dq|   (dk alike)
  dv       sum P (rP + U + g(n)) |do| + u |dv|
  dbias    sum eS + g(n) sum |dS| + u |dbias|
with a factor 1.05 for the products of errors; nothing is fitted.
"""
import numpy as np
import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from oracle.xattn import bucket_map, head_backward, head_forward, visible_keys
from tensor_model_transformer_tp_gb300 import functional as F

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EW = 2.0 ** -18
SLACK = 1.05


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def g_(K):
    return K * 2.0 ** -23


def f64(t):
    return t.detach().double().cpu().numpy()


def inside(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        bad = ~(same | (np.abs(got - want) <= SLACK * bound + 1e-30))
    assert not bad.any(), "%s: %d of %d off, first at %s (%r, want %r, bound %r)" % (
        what, bad.sum(), bad.size, np.argwhere(bad)[0], got[tuple(np.argwhere(bad)[0])],
        want[tuple(np.argwhere(bad)[0])], bound[tuple(np.argwhere(bad)[0])])


class Case:
    def __init__(self, dtype, B, Sq, Sk, H, G, D, lens=None, causal=False, start=None, buckets=0,
                 far=128, both=None, packed=True, scale=None, seed=0):
        self.dtype, self.B, self.Sq, self.Sk, self.H, self.G, self.D = dtype, B, Sq, Sk, H, G, D
        self.lens = [Sk] * B if lens is None else lens
        self.start = [start or 0] * B if not isinstance(start, list) else start
        self.causal, self.buckets, self.far = causal, buckets, far
        self.both = not causal if both is None else both
        self.scale = D ** -0.5 if scale is None else scale
        gen = torch.Generator().manual_seed(seed + B + 3 * Sq + 7 * Sk + 11 * H + 13 * D)

        def rnd(*shape, std=1.0):
            return (torch.randn(*shape, generator=gen) * std).to(T[dtype]).cuda()

        self.q = rnd(B, Sq, H, D)
        if packed:      # keys and values side by side in one projection
            kv = rnd(B, Sk, 2 * G, D)
            self.k, self.v = kv[:, :, :G], kv[:, :, G:]
        else:
            self.k, self.v = rnd(B, Sk, G, D), rnd(B, Sk, G, D)
        self.bias = rnd(buckets, H) if buckets else None
        self.do = rnd(B, Sq, H, D)
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        self.opt = dict(kv_lens=None if lens is None else ints(self.lens), causal=causal,
                        q_start=ints(start) if isinstance(start, list) else start,
                        scale=scale, bias=self.bias, max_distance=far, bidirectional=both)

    def forward(self):
        return F.attn_fwd(self.q, self.k, self.v, **self.opt)

    def backward(self, o, lse, **kw):
        return F.attn_bwd(self.q, self.k, self.v, o, lse, self.do, **self.opt, **kw)

    def check(self, o, lse, grads=None):
        u, Uo = U[self.dtype], U[self.dtype] if self.dtype == "bf16" else 0.0
        q, k, v, do, out = (f64(x) for x in (self.q, self.k, self.v, self.do, o))
        stat = f64(lse)
        if grads is not None:
            dq, dk, dv = (f64(x) for x in grads[:3])
            wk, wv, bk, bv = (np.zeros_like(dk) for _ in range(4))
            wb, bb, nb = (np.zeros((max(self.buckets, 1), self.H)) for _ in range(3))
        table = None if self.bias is None else f64(self.bias)
        sc = self.scale
        for b in range(self.B):
            n = self.lens[b]      # (what stands behind the keys may be anything)
            see = visible_keys(self.Sq, n, n, self.start[b], self.causal)
            if self.buckets:
                at = bucket_map(self.Sq, n, self.start[b], self.buckets, self.far, self.both)
            for h in range(self.H):
                g = h // (self.H // self.G)
                x, y, z, w = q[b, :, h], k[b, :n, g], v[b, :n, g], do[b, :, h]
                add = table[at, h] if self.buckets else None
                want, want_lse, P = head_forward(x, y, z, sc, add, see)
                mag = np.abs(add) if self.buckets else 0.0
                es = (g_(self.D) + 3 * 2.0 ** -23) * sc * (np.abs(x) @ np.abs(y).T) + \
                    3 * 2.0 ** -23 * mag
                es = np.where(see, es, 0.0)
                mean = (P * es).sum(axis=1, keepdims=True)
                rP = es + mean + EW
                keys = max(n, 1)
                eo = (P * (rP + Uo + g_(keys))) @ np.abs(z) + u * np.abs(want)
                tag = "b %d h %d" % (b, h)
                inside(out[b, :, h], want, eo, "o " + tag)
                some = ~np.isneginf(want_lse)
                assert (np.isneginf(stat[b, h]) == ~some).all(), "lse " + tag
                lb = mean[:, 0] + g_(keys) + EW + 2.0 ** -22 * np.abs(np.where(some, want_lse, 0.0))
                inside(stat[b, h][some], want_lse[some], lb[some], "lse " + tag)
                if grads is None:
                    continue
                ddq, ddk, ddv, dS = head_backward(x, y, z, P, w, sc)
                dP = w @ z.T
                delta = (P * dP).sum(axis=1, keepdims=True)
                ed = g_(self.D) * (np.abs(w) @ np.abs(z).T)
                et = (np.abs(w) * (eo + g_(self.D) * np.abs(want))).sum(axis=1, keepdims=True)
                eS = P * (rP * np.abs(dP - delta) + ed + et)
                rows = self.Sq * self.H // self.G
                inside(dq[b, :, h], ddq, sc * (eS + (Uo + g_(keys)) * np.abs(dS)) @ np.abs(y) +
                       u * np.abs(ddq), "dq " + tag)
                wk[b, :n, g] += ddk
                wv[b, :n, g] += ddv
                bk[b, :n, g] += sc * (eS + (Uo + g_(rows)) * np.abs(dS)).T @ np.abs(x)
                bv[b, :n, g] += (P * (rP + Uo + g_(rows))).T @ np.abs(w)
                if self.buckets:
                    for acc, val in ((wb, dS), (bb, eS), (nb, np.abs(dS))):
                        acc[:, h] += np.bincount(at.ravel(), val.ravel(), self.buckets)
        if grads is None:
            return
        inside(dk, wk, bk + u * np.abs(wk), "dk")
        inside(dv, wv, bv + u * np.abs(wv), "dv")
        if self.buckets:
            terms = g_(self.B * self.Sq * self.Sk)
            inside(grads[3], wb, bb + terms * nb + u * np.abs(wb), "dbias")
        else:
            assert grads[3] is None


def run(*a, **kw):
    c = Case(*a, **kw)
    o, lse = c.forward()
    grads = c.backward(o, lse)
    oz.oases_check_device(torch.cuda.current_stream())
    c.check(o, lse, grads)
    return c, o, lse, grads


# (batch, queries, keys, heads, key heads, head size)
SHAPES = [(1, 1, 1, 1, 1, 8), (2, 1, 300, 4, 2, 64), (3, 5, 77, 2, 2, 32), (1, 64, 64, 2, 1, 128),
          (2, 127, 129, 2, 2, 40), (1, 128, 128, 1, 1, 64), (1, 130, 259, 4, 1, 72),
          (2, 300, 65, 2, 2, 16), (1, 257, 513, 2, 1, 128), (1, 63, 700, 3, 3, 96),
          (1, 520, 130, 2, 2, 128), (1, 385, 384, 1, 1, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_keys_of_another_length(dtype, shape):
    run(dtype, *shape)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
def test_ragged_keys(dtype, shape):
    """Lengths 0, 1, odd ones and the whole; the last queries' sequences among them."""
    B, Sq, Sk, H, G, D = shape
    for lens in ([0, 1, Sk], [Sk, max(0, Sk - 1), 0], [Sk // 2, Sk // 3, 1]):
        run(dtype, 3, Sq, Sk, H, G, D, lens=lens)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq,Sk,start", [(1, 200, [0, 150, 199]), (40, 200, [0, 100, 160]),
                                         (200, 200, None), (300, 140, None), (130, 400, 270),
                                         (257, 300, [43, 0, 7]), (70, 70, 500)])
def test_causal(dtype, Sq, Sk, start):
    run(dtype, 3, Sq, Sk, 2, 1, 64, causal=True, start=start)
    run(dtype, 3, Sq, Sk, 2, 2, 128, causal=True, start=start, lens=[Sk, Sk // 2, 0])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq,Sk,causal,buckets,far,both,D", [
    (130, 130, False, 32, 128, True, 64), (300, 300, True, 32, 128, False, 64),
    (400, 400, False, 16, 20, True, 128), (600, 600, False, 32, 30, True, 40),
    (257, 700, False, 64, 250, True, 64), (300, 200, True, 128, 300, False, 128),
    (1, 400, True, 32, 128, False, 64), (65, 65, False, 8, 400, False, 32),
    (530, 530, True, 2, 2, False, 64), (200, 500, True, 32, 64, True, 96)])
def test_position_bias(dtype, Sq, Sk, causal, buckets, far, both, D):
    start = Sk - Sq if Sk > Sq else 0
    kw = dict(causal=causal, buckets=buckets, far=far, both=both, scale=1.0 / D)
    run(dtype, 1, Sq, Sk, 2, 1, D, start=start, **kw)
    run(dtype, 3, Sq, Sk, 2, 2, D, start=[0, start, start // 2], lens=[Sk, Sk // 3, 0], **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("biased", [False, True])
def test_whatever_stands_behind_the_keys(dtype, biased):
    """NaN and infinities at and behind kv_lens change nothing."""
    kw = dict(lens=[131, 1, 64], buckets=32 if biased else 0, packed=False)
    for Sq, D in ((1, 64), (150, 64), (200, 128)):
        c = Case(dtype, 3, Sq, 200, 2, 1, D, **kw)
        o, lse = c.forward()
        first = (o, lse, *c.backward(o, lse))
        for b, n in enumerate(c.lens):
            c.k[b, n:] = float("nan")
            c.v[b, n:] = float("inf")
            c.v[b, n + 3:] = float("nan")
        o, lse = c.forward()
        for x, y in zip(first, (o, lse, *c.backward(o, lse))):
            assert x is y is None or torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_biases_that_hide_keys(dtype):
    """-inf hides a bucket's keys; the type's lowest value hides them beside others and
    counts them alone; a query all of whose keys are hidden has no output."""
    for value, Sq in ((float("-inf"), 150), (torch.finfo(T[dtype]).min, 150),
                      (float("-inf"), 1), (torch.finfo(T[dtype]).min, 1)):
        c = Case(dtype, 1, Sq, 150, 2, 2, 64, buckets=32, causal=True, start=0)
        c.bias[0] = value           # the query's own position
        o, lse = c.forward()
        dq, dk, dv, db = c.backward(o, lse)
        if value == float("-inf"):
            assert not o[:, 0].any() and torch.isneginf(lse[:, :, 0]).all()
            assert not dq[:, 0].any() and not db[0].any()
        else:                       # query 0 sees key 0 alone
            assert torch.equal(o[:, 0], c.v[:, 0])
        assert all(torch.isfinite(x).all() for x in (o, dq, dk, dv, db))
        if Sq > 1:
            c.bias[0] = -1e4        # (a finite stand-in of the same weight, 0)
            p, lse_p = c.forward()
            grads = c.backward(p, lse_p)
            assert torch.equal(o[:, 1:], p[:, 1:]) and torch.equal(dq[:, 1:], grads[0][:, 1:])
            assert torch.equal(db[1:], grads[3][1:])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_layouts(dtype):
    """Packed projections, transposed heads, gradients into slices of one buffer: the
    same bits as contiguous tensors."""
    B, S, H, D = 2, 150, 2, 64
    c = Case(dtype, B, S, S, H, H, D, causal=True, buckets=32, packed=False)
    o, lse = c.forward()
    want = (o, lse, *c.backward(o, lse))
    qkv = torch.cat([c.q, c.k, c.v], dim=2)
    grads = torch.full_like(qkv, float("nan"))
    views = [qkv[:, :, i * H:(i + 1) * H] for i in range(3)]
    out = [grads[:, :, i * H:(i + 1) * H] for i in range(3)]
    o, lse = F.attn_fwd(*views, **c.opt)
    got = F.attn_bwd(*views, o, lse, c.do, **c.opt, out=out)
    assert all(g is t for g, t in zip(got, out))
    for x, y in zip(want, (o, lse, *got)):
        assert torch.equal(x, y)
    heads_first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (c.q, c.k, c.v)]
    tokens_first = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in heads_first]
    for views in (heads_first, tokens_first):
        o, lse = F.attn_fwd(*views, **c.opt)
        do = c.do.transpose(1, 2).contiguous().transpose(1, 2)
        o2 = o.transpose(0, 1).contiguous().transpose(0, 1)
        for x, y in zip(want, (o, lse, *F.attn_bwd(*views, o2, lse, do, **c.opt))):
            assert torch.equal(x, y)


def test_accumulated_and_left_out_bias_gradient():
    for dtype in T:
        c = Case(dtype, 2, 140, 140, 2, 2, 64, buckets=32)
        o, lse = c.forward()
        first = c.backward(o, lse)
        acc = torch.full((32, 2), 3.0, device="cuda")
        got = c.backward(o, lse, dbias=acc)
        assert got[3] is acc
        zero = torch.zeros_like(acc)
        c.backward(o, lse, dbias=zero)
        assert torch.equal(acc, zero + 3.0) and torch.equal(zero.to(T[dtype]), first[3])
        none = c.backward(o, lse, need_dbias=False)
        assert none[3] is None and all(torch.equal(a, b) for a, b in zip(none[:3], first[:3]))


def test_empty_batches_and_lengths():
    for dtype in T:
        for B, Sq, Sk in ((0, 5, 7), (2, 0, 7), (2, 5, 0)):
            c = Case(dtype, B, Sq, Sk, 2, 1, 64, buckets=32)
            o, lse = c.forward()
            assert not o.any() and torch.isneginf(lse).all()
            dq, dk, dv, db = c.backward(o, lse)
            assert not dq.any() and not dk.any() and not dv.any() and not db.any()


def test_captured_replayed_and_on_another_stream():
    """A captured training pass gives an eager one's bits, also replayed on new inputs,
    also on another stream while the first runs."""
    for dtype, kw in (("bf16", dict(buckets=32, causal=True, lens=[150, 33])), ("bf16", {}),
                      ("f32", dict(buckets=32))):
        for Sq in (1, 150):
            c = Case(dtype, 2, Sq, 150, 4, 2, 64, **kw)
            o, lse = c.forward()
            want = (o, lse, *c.backward(o, lse))
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                o, lse = c.forward()
                other = (o, lse, *c.backward(o, lse))
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, lse = c.forward()
                got = (o, lse, *c.backward(o, lse))
            for _ in range(2):
                for t in got:
                    if t is not None:
                        t.fill_(float("nan"))
                graph.replay()
            torch.cuda.synchronize()
            for x, y, z in zip(want, got, other):
                assert x is y is z is None or (torch.equal(x, y) and torch.equal(x, z))
            c.q.mul_(0.5)
            graph.replay()
            o, lse = c.forward()
            for x, y in zip((o, lse, *c.backward(o, lse)), got):
                assert x is y is None or torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq,Sk,causal", [(1, 1, False), (150, 1, False), (200, 200, True), (3, 400, False)])
def test_a_single_key_gives_no_gradient(dtype, Sq, Sk, causal):
    """Of weight 1 whatever its score: dq, dk and dbias are 0, not what roundings leave."""
    lens = [Sk, 1]
    c, o, lse, (dq, dk, dv, db) = run(dtype, 2, Sq, Sk, 4, 2, 64, lens=lens, causal=causal, buckets=16)
    assert not dq[1].any() and not dk[1].any()
    assert torch.equal(o[1, :, 2], c.v[1, :1, 1].expand(Sq, -1))
    if causal:
        assert not dq[0, 0].any()
    if Sk == 1:
        assert not dq.any() and not dk.any() and not db.any()


@pytest.mark.parametrize("Sq,Sk", [(300, 3), (130, 40), (257, 128), (400, 400)])
def test_delta_is_that_of_the_weights(Sq, Sk):
    """Rows of few keys, where delta of the rounded o would show: what remains is the
    rounding of dS and of dq, at most half a step of bf16 each, so that the norm of the
    error is at most 2 u |dq| and, the roundings' signs being random, near 1.4 u / sqrt(3);
    dbias has its own rounding alone."""
    c = Case("bf16", 2, Sq, Sk, 2, 2, 64, buckets=32, causal=Sq == Sk)
    o, lse = c.forward()
    dq, dk, dv, db = c.backward(o, lse)
    wide = {n: getattr(c, n).double().requires_grad_(True) for n in ("q", "k", "v", "bias")}
    s = torch.einsum("bihd,bjhd->bhij", wide["q"], wide["k"]) * c.scale
    at = torch.tensor(bucket_map(Sq, Sk, 0, 32, 128, c.both), device="cuda")
    s = s + wide["bias"][at].permute(2, 0, 1)
    if c.causal:
        see = torch.tensor(visible_keys(Sq, Sk, Sk, 0, True), device="cuda")
        s = s.masked_fill(~see, float("-inf"))
    want = torch.autograd.grad(torch.einsum("bhij,bjhd->bihd", torch.softmax(s, -1), wide["v"]),
                               [wide["q"], wide["k"], wide["bias"]], c.do.double())
    u = 2.0 ** -8
    for got, w, most in ((dq, want[0], 2 * u), (dk, want[1], 2 * u), (db, want[2], u)):
        assert (got.double() - w).norm() <= most * w.norm() * 1.05


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq", [1, 140])
def test_a_nan_shows(dtype, Sq):
    """A query of NaN has a NaN for an output, beside others that have none."""
    c = Case(dtype, 1, Sq, 200, 2, 1, 64)
    c.q[0, Sq // 2, 1] = float("nan")
    o, lse = c.forward()
    bad = torch.zeros(1, Sq, 2, dtype=torch.bool, device="cuda")
    bad[0, Sq // 2, 1] = True
    assert torch.equal(o.isnan().all(-1), bad) and torch.equal(o.isnan().any(-1), bad)
    assert torch.equal(lse.isnan(), bad.transpose(1, 2))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [-1e30, -1e9, -3e7])
def test_scores_beyond_what_weights_resolve_give_no_gradient(dtype, value):
    """A bias that hides every key by a finite value: no gradient, and none of it infinite."""
    c = Case(dtype, 1, 150, 150, 2, 2, 64, buckets=32)
    c.bias[:, 1] = value
    o, lse = c.forward()
    dq, dk, dv, db = c.backward(o, lse)
    assert all(torch.isfinite(x).all() for x in (o, lse, dq, dk, dv, db))
    assert not dq[:, :, 1].any() and not dk[:, :, 1].any() and not db[:, 1].any()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_many_ragged_sequences(causal, D):
    """Sequences in another order of length than of place, some empty, some alike."""
    lens = [0, 300, 17, 300, 129, 256, 1, 0, 270]
    run("bf16", 9, 200, 300, 4, 2, D, lens=lens, causal=causal, start=[0, 100, 3, 99, 0, 57, 0, 0, 71] if causal else 0,
        buckets=16)


@pytest.mark.parametrize("Sq", [1, 5])
def test_more_ragged_sequences_than_are_ordered(Sq):
    run("bf16", 270, Sq, 140, 2, 2, 40, lens=[(37 * b) % 141 for b in range(270)])


# few items over long keys or many queries, whose backward cuts them into pieces
CUT = [(1, 70, 2100, 2, 1, 64), (2, 1300, 70, 4, 2, 64), (1, 70, 1500, 1, 1, 128),
       (1, 1300, 150, 2, 1, 128), (3, 900, 1200, 4, 4, 40)]


@pytest.mark.parametrize("shape", CUT)
@pytest.mark.parametrize("biased", [False, True])
def test_items_in_pieces(shape, biased):
    lens = [shape[2] - shape[2] // 3 * b for b in range(shape[0])]
    run("bf16", *shape, lens=lens, buckets=32 if biased else 0)


@pytest.mark.parametrize("D", [64, 128])
def test_whole_rounds_and_pieces(D):
    """More items than SMs, the last of them cut: 200 of dq, 160 of dk and dv."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    run("bf16", 1, 1100, 1100, sms // 9 + 4, sms // 9 + 4, D, buckets=16, causal=True)


def test_many_sequences_and_heads():
    """More (sequence, head) pairs than SMs, ragged, with splits of long keys."""
    c = Case("bf16", 40, 3, 500, 8, 2, 64, lens=[(37 * i) % 501 for i in range(40)], causal=True,
             start=[max(0, (37 * i) % 501 - 3) for i in range(40)], buckets=32)
    o, lse = c.forward()
    c.check(o, lse, c.backward(o, lse))


def test_few_queries_over_long_keys():
    for dtype in T:
        for Sq, H, G in ((1, 2, 2), (2, 4, 1), (17, 2, 1), (64, 1, 1)):
            c = Case(dtype, 1, Sq, 5003, H, G, 64, buckets=32, far=600, start=2500)
            o, lse = c.forward()
            c.check(o, lse)
            c = Case(dtype, 2, Sq, 4100, H, G, 128, lens=[4099, 1290])
            o, lse = c.forward()
            c.check(o, lse, c.backward(o, lse))


@pytest.mark.parametrize("shape", [(1, 700, 60, 2, 1, 64), (1, 40, 900, 1, 1, 40), (2, 600, 300, 2, 1, 128),
                                   (1, 1500, 1500, 16, 16, 32)])
@pytest.mark.parametrize("biased", [False, True])
def test_shares_of_fp32(shape, biased):
    """Few tiles over many blocks, and tiles of 64 rows (the last)."""
    run("f32", *shape, lens=[shape[2] - 5 * b for b in range(shape[0])], buckets=48 if biased else 0,
        causal=shape[1] == shape[2])


@pytest.mark.parametrize("dtype,most", [("f32", 2e-3), ("bf16", 0.15)])
def test_a_layer_of_one_projection(dtype, most):
    """Norms and rotation, attention, and both backward into slices of one packed gradient,
    against autograd in 64 bits.  In fp32 each of six stages is off by g(K) = K 2^-23 at most,
    K <= 100 terms, which the softmax (scores up to 8) multiplies by 16 at most: 1.2e-3.  In
    bf16 the rounded q' and k' move a score by 2 u sqrt(D) at most, a weight by twice that, and
    five more roundings add u each: 0.14 of the gradients' norm."""
    B, S, H, G, D, R = 3, 100, 4, 2, 64, 32
    gen = torch.Generator().manual_seed(5)
    make = lambda *shape: torch.randn(*shape, generator=gen).to(T[dtype]).cuda()  # noqa: E731
    qkv, wq, wk, do = make(B, S, H + 2 * G, D), make(D), make(D), make(B, S, H, D)
    bias = make(16, H)
    lens = torch.tensor([100, 37, 64], dtype=torch.int32, device="cuda")
    angle = torch.arange(S, device="cuda")[:, None] * 100.0 ** (-torch.arange(R // 2, device="cuda") / (R // 2))
    cos, sin = angle.cos().float(), angle.sin().float()
    q, k, v = qkv[:, :, :H], qkv[:, :, H:H + G], qkv[:, :, H + G:]
    opt = dict(kv_lens=lens, causal=True, bias=bias)
    q2, k2 = F.qk_norm_rope_fwd(q, k, cos, sin, q_weight=wq, k_weight=wk)
    o, lse = F.attn_fwd(q2, k2, v, **opt)
    grad = torch.empty_like(qkv)
    dq, dk, dv = grad[:, :, :H], grad[:, :, H:H + G], grad[:, :, H + G:]
    _, _, _, db = F.attn_bwd(q2, k2, v, o, lse, do, out=(dq, dk, dv), **opt)
    _, _, dwq, dwk = F.qk_norm_rope_bwd(q, k, dq, dk, cos, sin, q_weight=wq, k_weight=wk, out=(dq, dk))
    oz.oases_check_device(torch.cuda.current_stream())

    wide = [x.double().requires_grad_(True) for x in (qkv, wq, wk, bias)]

    def turned(x, w):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b, rest = x[..., :R // 2], x[..., R // 2:R], x[..., R:]
        c, s = cos.double()[None, :, None], sin.double()[None, :, None]
        return torch.cat([a * c - b * s, a * s + b * c, rest], -1)

    Q = turned(wide[0][:, :, :H], wide[1])
    K, V = turned(wide[0][:, :, H:H + G], wide[2]), wide[0][:, :, H + G:]
    at = torch.tensor(bucket_map(S, S, 0, 16, 128, False), device="cuda")
    s = torch.einsum("bihd,bjhd->bhij", Q, K.repeat_interleave(H // G, 2)) * D ** -0.5 + wide[3][at].permute(2, 0, 1)
    n = torch.arange(S, device="cuda")
    s = s.masked_fill((n[None] > n[:, None]) | (n >= lens[:, None, None, None]), float("-inf"))
    want_o = torch.einsum("bhij,bjhd->bihd", torch.softmax(s, -1), V.repeat_interleave(H // G, 2))
    want = torch.autograd.grad(want_o, wide, do.double())
    for got, w in ((o, want_o.detach()), (grad, want[0]), (dwq, want[1]), (dwk, want[2]), (db, want[3])):
        assert (got.double() - w).norm() <= most * w.norm()
