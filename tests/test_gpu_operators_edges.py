"""Edges of the gated feed-forward block (oases_glu.h) and the linear head's cross
entropy (oases_ce.h) on the GPU: values and sizes at the ends of what the headers
allow."""
import itertools

import numpy as np
import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from tensor_model_transformer_tp_gb300 import functional as F

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def ce_tensors(dtype, M, H, V, seed=0):
    gen = torch.Generator().manual_seed(seed + M + 3 * H + 5 * V)
    x = torch.randn(M, H, generator=gen).to(T[dtype]).cuda()
    w = (torch.randn(V, H, generator=gen) * H ** -0.5).to(T[dtype]).cuda()
    t = torch.randint(0, V, (M,), generator=gen)
    t[::3] = -100
    return x, w, t.cuda()


# ---- one dloss for all rows that is infinite or NaN ------------------------------
# (37 x 40000: dx in split parts; 8000 x 20001: several pieces of the vocabulary)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype,M,H,V", [("bf16", 12, 64, 300), ("bf16", 140, 72, 901),
                                         ("bf16", 37, 64, 40000), ("bf16", 8000, 64, 20001),
                                         ("f32", 12, 33, 301), ("f32", 140, 64, 900)])
def test_ce_non_finite_dloss_of_all_rows_stays_in_the_rows_with_a_loss(dtype, M, H, V, value):
    x, w, t = ce_tensors(dtype, M, H, V)
    d = torch.full((1,), value, device="cuda")
    _, lse = F.ce_fwd(x, w, t)
    dx, dw = F.ce_bwd(x, w, t, lse, d)
    ignored = t == -100
    assert not dx[ignored].any()                         # 0, not NaN
    assert not torch.isfinite(dx[~ignored]).any() and not torch.isfinite(dw).any()
    # every row ignored (the mean over no rows: 1 / 0): no gradient at all
    none = torch.full_like(t, -100)
    start = torch.randn_like(w, dtype=torch.float32)
    acc = start.clone()
    dx, dw = F.ce_bwd(x, w, none, lse, d)
    assert not dx.any() and not dw.any()
    dx, _ = F.ce_bwd(x, w, none, lse, d, dw=acc)
    assert not dx.any() and torch.equal(acc, start)
