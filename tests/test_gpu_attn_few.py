"""Attention over keys of another length on the GPU: the forward for a few query rows a key
head, all of its row counts, against the definition and bounds of test_gpu_attn.py, and
calls that are under way together."""
import threading

import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from tensor_model_transformer_tp_gb300 import functional as F
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def forward(*a, **kw):
    c = Case(*a, **kw)
    o, lse = c.forward()
    oz.oases_check_device(torch.cuda.current_stream())
    c.check(o, lse)


# (queries, heads, key heads): 1 to 4 rows of a key head, those of several queries among them,
# and the first beyond
ROWS = [(1, 2, 2), (1, 4, 2), (2, 3, 3), (1, 3, 1), (3, 2, 2), (1, 8, 2), (2, 4, 2), (4, 1, 1), (5, 1, 1), (1, 8, 1)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D", [8, 64, 72, 128])
@pytest.mark.parametrize("rows", ROWS)
def test_rows_of_a_key_head(dtype, D, rows):
    """Ragged and whole, causal behind a cache and not: a step's odd end, one key, none."""
    Sq, H, G = rows
    forward(dtype, 2, Sq, 333, H, G, D)
    forward(dtype, 5, Sq, 257, H, G, D, lens=[257, 0, 1, 130, 64])
    forward(dtype, 4, Sq, 300, H, G, D, lens=[300, 77, 5, 300], causal=True, start=[296, 73, 0, -2])
    forward(dtype, 1, Sq, 1, H, G, D)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("buckets,far,both", [(32, 128, False), (32, 700, True), (64, 250, True), (3, 2, False)])
def test_rows_of_a_key_head_with_a_bias(dtype, rows, buckets, far, both):
    """By distance from a table (borders up to 256) and searched for (beyond)."""
    Sq, H, G = rows
    kw = dict(buckets=buckets, far=far, both=both, scale=1 / 64)
    forward(dtype, 3, Sq, 900, H, G, 64, lens=[900, 411, 0], start=[450, 411 - Sq, 0], **kw)
    forward(dtype, 2, Sq, 1100, H, G, 40, lens=[1100, 513], causal=True, start=[1100 - Sq, 200], **kw)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [(1, 4, 1), (3, 1, 1), (1, 2, 1), (1, 16, 1)])
def test_long_keys_of_few_sequences(dtype, rows):
    """Shares joined within a cluster and through memory."""
    Sq, H, G = rows
    forward(dtype, 1, Sq, 9001, H, G, 128, start=8990, causal=True)
    forward(dtype, 3, Sq, 6000, H, G, 64, lens=[6000, 17, 3001], buckets=32, start=[5000, 17, 3000])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("threads", [False, True])
def test_passes_under_way_together(dtype, threads):
    """Training passes and single tokens on two streams, from one thread or two, with no order
    between them: each has the bits that it has alone."""
    shapes = [dict(B=3, Sq=150, Sk=150, H=4, G=2, D=64, causal=True, buckets=32, lens=[150, 33, 90]),
              dict(B=2, Sq=130, Sk=700, H=2, G=1, D=128),
              dict(B=4, Sq=1, Sk=3000, H=4, G=2, D=64, buckets=16, start=2000)]
    work = [[Case(dtype, seed=s, **kw) for kw in shapes] for s in (1, 2)]

    def once(c):
        o, lse = c.forward()
        return [o, lse, *c.backward(o, lse)]

    want = [[once(c) for c in cases] for cases in work]
    torch.cuda.synchronize()
    got, failed = [[], []], []

    def drive(i, rounds):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(rounds):
                    got[i].append([once(c) for c in work[i]])
        except Exception as e:
            failed.append(e)

    streams = [torch.cuda.Stream() for _ in work]
    if threads:
        both = [threading.Thread(target=drive, args=(i, 12)) for i in range(2)]
        for t in both:
            t.start()
        for t in both:
            t.join()
    else:
        for _ in range(12):
            for i in range(2):
                drive(i, 1)
    torch.cuda.synchronize()
    assert not failed
    for i in range(2):
        assert len(got[i]) == 12
        for result in got[i]:
            for c, w in zip(result, want[i]):
                assert all(x is y is None or torch.equal(x, y) for x, y in zip(c, w))


def test_two_graphs_under_way_together():
    """Two captured passes, replayed side by side on two streams on changing inputs."""
    cases = [Case("bf16", 3, 150, 150, 4, 2, 64, causal=True, buckets=32, lens=[150, 33, 90], seed=s) for s in (1, 2)]

    def once(c):
        o, lse = c.forward()
        return [o, lse, *c.backward(o, lse)]

    once(cases[0])
    graphs, got = [], []
    for c in cases:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(once(c))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(3):
        for c in cases:
            c.q.mul_(-0.5)
        torch.cuda.synchronize()
        for _ in range(10):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for c, r in zip(cases, got):
            assert all(torch.equal(x, y) for x, y in zip(r, once(c)))


def test_norms_under_way_together():
    """Norms and rotation, forward and backward, on two streams with no order between them."""
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *shape: torch.randn(*shape, generator=gen).cuda().bfloat16()  # noqa: E731
    cos, sin = (torch.randn(500, 32, generator=gen).cuda() for _ in range(2))
    data = [[rnd(4, 500, 8, 64), rnd(4, 500, 2, 64), rnd(4, 500, 8, 64), rnd(4, 500, 2, 64), rnd(64), rnd(64)]
            for _ in range(2)]

    def once(q, k, dq, dk, wq, wk):
        opt = dict(q_weight=wq, k_weight=wk)
        return [*F.qk_norm_rope_fwd(q, k, cos, sin, **opt), *F.qk_norm_rope_bwd(q, k, dq, dk, cos, sin, **opt)]

    want = [once(*d) for d in data]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in data], [[], []]
    for _ in range(20):
        for i, d in enumerate(data):
            with torch.cuda.stream(streams[i]):
                got[i].append(once(*d))
    torch.cuda.synchronize()
    for i in range(2):
        for result in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(result, want[i]))
