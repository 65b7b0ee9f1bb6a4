"""Attention over keys of another length (oases_attn.h) on the GPU at sizes and starts
beside those of test_gpu_attn.py, whose definition and bounds these tests use."""
import copy

import numpy as np
import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from oracle.xattn import bucket_map
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def heads_of(c, first, end):
    """The case of some of c's heads (as many key heads as query heads)."""
    part = copy.copy(c)
    part.H = part.G = end - first
    part.q, part.k, part.v, part.do = (x[:, :, first:end] for x in (c.q, c.k, c.v, c.do))
    part.bias = c.bias[:, first:end]
    return part


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq", [1, 5])
def test_more_heads_with_a_bias_than_a_grid_is_wide(dtype, Sq):
    """65536 and more, each with a bias of its own (and, of one query, more pairs of sequence
    and key head than the kernel for single tokens takes)."""
    H = 65536 + 24
    c = Case(dtype, 1, Sq, 7, H, H, 8, buckets=4, far=3)
    o, lse = c.forward()
    dq, dk, dv, db = c.backward(o, lse)
    oz.oases_check_device(torch.cuda.current_stream())
    for first, end in ((0, 8), (32760, 32776), (65528, 65544), (H - 8, H)):
        heads_of(c, first, end).check(o[:, :, first:end], lse[:, first:end],
                                      [x[:, :, first:end] for x in (dq, dk, dv)] + [db[:, first:end]])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("Sq,Sk,start", [(200, 201, 1), (150, 250, [100, 1, 50]), (128, 1100, [100, 127, 64]),
                                         (300, 200, [-100, -1, -257])])
def test_delta_of_few_keys_behind_a_start(Sq, Sk, start, biased, D):
    """Queries that see 128 keys or less beside others, of the same tile, that see more.  Their
    values of v are 1 + noise / 16, so that delta from the rounded o would be off by up to
    u |dO| sqrt(D) where dP - delta is |dO| sqrt(D) / 16 in size: 0.0625 / sqrt(3) of dS, nine
    times what may remain.  That is the rounding of dS and of dq (of dk), half a step each: the norm
    of the error is at most 2 u of the gradient's.  The other queries have no dO."""
    B = 3
    c = Case("bf16", B, Sq, Sk, 4, 2, D, causal=True, start=start if isinstance(start, list) else [start] * B,
             buckets=16 if biased else 0, far=100)
    c.v.mul_(1 / 16).add_(1.0)
    seen = torch.tensor(c.start, device="cuda")[:, None] + torch.arange(1, Sq + 1, device="cuda")    # [B, Sq]
    c.do[seen > 128] = 0.0
    o, lse = c.forward()
    dq, dk, dv, db = c.backward(o, lse)
    oz.oases_check_device(torch.cuda.current_stream())
    wide = {n: getattr(c, n).double().requires_grad_(True) for n in ["q", "k", "v"] + ["bias"] * biased}
    k, v = (wide[n].repeat_interleave(2, dim=2) for n in "kv")
    s = torch.einsum("bihd,bjhd->bhij", wide["q"], k) * c.scale
    if biased:
        at = torch.tensor(np.stack([bucket_map(Sq, Sk, p, 16, 100, False) for p in c.start]), device="cuda")
        s = s + wide["bias"][at].permute(0, 3, 1, 2)
    hide = (torch.arange(Sk, device="cuda")[None, None] >= seen[:, :, None])[:, None]
    none = hide.all(-1, keepdim=True)
    P = torch.softmax(s.masked_fill(hide, float("-inf")).masked_fill(none, 0.0), -1).masked_fill(none, 0.0)
    want = torch.autograd.grad(torch.einsum("bhij,bjhd->bihd", P, v), list(wide.values()), c.do.double())
    u = 2.0 ** -8
    got = [dq, dk, dv] + [db] * biased
    for name, x, w, most in zip(("dq", "dk", "dv", "dbias"), got, want, (2 * u, 2 * u, 2 * u, u)):
        assert (x.double() - w).norm() <= most * w.norm() * 1.05, name


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("value", [3e7, 1e9, 1e30, "max"])
def test_scores_above_what_weights_resolve_give_no_gradient(dtype, value):
    """As those far below: from a bias that lifts every key of head 1 comes no gradient, and
    none of it infinite; the output is that without a bias, and head 0's has its own."""
    c = Case(dtype, 1, 150, 150, 2, 2, 64, buckets=32)
    c.bias[:, 1] = 0.0
    plain, _ = c.forward()
    c.bias[:, 1] = torch.finfo(c.bias.dtype).max if value == "max" else value
    o, lse = c.forward()
    dq, dk, dv, db = c.backward(o, lse)
    assert all(torch.isfinite(x).all() for x in (o, lse, dq, dk, dv, db))
    assert torch.equal(o[:, :, 0], plain[:, :, 0])
    for x in (dq[:, :, 1], dk[:, :, 1], dv[:, :, 1], db[:, 1]):
        assert not x.any()
    assert dq[:, :, 0].any() and dv[:, :, 0].any() and db[:, 0].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Sq,H,D", [(1, 2, 64), (1, 8, 64), (5, 1, 128), (40, 2, 64), (150, 2, 128), (300, 1, 40)])
@pytest.mark.parametrize("biased", [False, True])
def test_whatever_stands_behind_the_last_query(dtype, Sq, H, D, biased):
    """Causal over a cache that is not full, no kv_lens: NaN and infinities behind a sequence's
    last query, where none sees them, change nothing."""
    start = [0, 37, 120, -Sq, 500 - Sq]
    c = Case(dtype, 5, Sq, 500, H, 1, D, causal=True, start=start, buckets=32 if biased else 0, packed=False)
    for b, p in enumerate(start):
        c.k[b, p + Sq:] = 0.0
        c.v[b, p + Sq:] = 0.0
    o, lse = c.forward()
    first = (o, lse, *c.backward(o, lse))
    c.check(o, lse, first[2:])
    for b, p in enumerate(start):
        c.k[b, p + Sq:] = float("nan")
        c.v[b, p + Sq:] = float("inf")
        c.v[b, p + Sq + 3:] = float("nan")
    o, lse = c.forward()
    for x, y in zip(first, (o, lse, *c.backward(o, lse))):
        assert x is y is None or torch.equal(x, y)
