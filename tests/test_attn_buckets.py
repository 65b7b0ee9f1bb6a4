"""The buckets of relative positions as the library has them (oases_attn.h): every border
against the definition in whole numbers (oracle/xattn.py), and the cost of finding them."""
import ctypes
import time

import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from oracle.xattn import bucket
from tensor_model_transformer_tp_gb300 import functional as F


@pytest.fixture(scope="module", autouse=True)
def _library():
    oz.build_library()


def check_time(buckets):
    """Seconds of the library's check of a descriptor (a size query of an empty call), the
    least of many."""
    strides = {n: oz.Strides(128, 64, 64) for n in ("q", "k", "v", "o")}
    d = oz.AttnDesc(dtype=1, batch=2, q_len=0, k_len=1, heads=1, kv_heads=1, head_dim=64, causal=1,
                    buckets=buckets, max_distance=1000, bidirectional=0, scale=1.0, **strides)
    query, at = oz.lib().oases_attn_workspace_bytes, ctypes.byref(d)
    least = float("inf")
    for _ in range(300):
        t = time.perf_counter()
        for _ in range(10):
            query(at, 0)
        least = min(least, (time.perf_counter() - t) / 10)
    return least


def test_borders_cost_a_call_nothing():
    """Every call of the library finds the borders anew: by doubles, without memory of the
    heap's and without powers of hundreds of digits but where a border is a whole number."""
    assert check_time(128) < check_time(0) + 10e-6


@pytest.mark.gpu
@pytest.mark.parametrize("buckets,far,both", [
    (32, 128, True), (32, 128, False), (16, 64, True), (8, 5, False), (4, 100, True), (64, 250, False),
    (2, 2, False), (128, 65536, False), (128, 65536, True), (128, 65, False), (128, 16384, False), (3, 7, False),
    (33, 4096, False), (64, 8192, True), (100, 12345, False), (5, 65536, False)])
def test_every_bucket_is_the_definition(buckets, far, both):
    """A query over the one key at position 0 has lse = the bias of its distance: with the
    table's rows their own numbers (to within 2^-20 of them, so rounded), the bucket."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    S = far + 50
    table = torch.arange(buckets, device="cuda", dtype=torch.float32)[:, None].contiguous()
    q, k = torch.zeros(2, S, 1, 8, device="cuda"), torch.zeros(2, 1, 1, 8, device="cuda")
    start = torch.tensor([0, 1 - S], dtype=torch.int32, device="cuda")       # n = 0, -1, .. and S - 1, ..
    _, lse = F.attn_fwd(q, k, k, bias=table, max_distance=far, bidirectional=both, q_start=start)
    past, ahead = lse[:, 0].round().long().tolist()
    for side, sign in ((past, -1), (ahead[::-1], 1)):
        # the definition's buckets rise with the distance: right on both sides of every step
        # of the library's is right throughout
        steps = [a for a in range(1, S) if side[a] != side[a - 1]]
        for a in sorted({0, S - 1, *steps, *(a - 1 for a in steps)}):
            assert side[a] == bucket(sign * a, buckets, far, both), (a, sign)
