"""Arguments of the functions on torch tensors that no library call could carry,
refused without a GPU: shapes are given as the signatures the plans are checked
against (shape, type, CUDA device)."""
import warnings

import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from tensor_model_transformer_tp_gb300 import functional as F

BF, BIG = torch.bfloat16, (1 << 32) + 8


@pytest.fixture(scope="module", autouse=True)
def _library():
    oz.build_library()


def sig(*shape, dtype=BF):
    return torch.Size(shape), dtype, 0


def glu_sigs(rows=4, hidden=64, ffn=128):
    return sig(rows, hidden), (sig(2 * ffn, hidden), None, sig(hidden, ffn), None)


@pytest.mark.parametrize("size", [BIG, 1 << 31])
@pytest.mark.parametrize("name", ["rows", "hidden", "ffn"])
def test_glu_sizes_beyond_32_bits(name, size):
    """2^32 + 8 rows are not 8 rows."""
    x, w = glu_sigs(**{name: size})
    with pytest.raises(ValueError, match=name):
        F._glu_fwd_plan(x, w, None, None, "silu", "none")
    with pytest.raises(ValueError, match=name):
        F._glu_bwd_plan(x, w, x, None, None, "silu", "none", None)


@pytest.mark.parametrize("size", [BIG, 1 << 31])
@pytest.mark.parametrize("name", ["rows", "hidden", "vocab"])
def test_ce_sizes_beyond_32_bits(name, size):
    n = {"rows": 4, "hidden": 64, "vocab": 100, name: size}
    x, w = sig(n["rows"], n["hidden"]), sig(n["vocab"], n["hidden"])
    t, f = sig(n["rows"], dtype=torch.int64), sig(n["rows"], dtype=torch.float32)
    with pytest.raises(ValueError, match=name):
        F._ce_plan(x, w, t, None, None, None, False, -100)
    with pytest.raises(ValueError, match=name):
        F._ce_plan(x, w, t, f, f, None, True, -100)


@pytest.mark.parametrize("index", [1 << 63, (1 << 64) - 100, -(1 << 63) - 1])
def test_ce_ignore_index_beyond_64_bits(index):
    """2^64 - 100 is not -100."""
    x, w, t = sig(4, 64), sig(100, 64), sig(4, dtype=torch.int64)
    with pytest.raises(ValueError, match="ignore_index"):
        F._ce_plan(x, w, t, None, None, None, False, index)


# ---- tensors that autograd follows ---------------------------------------------------
def test_a_forward_that_autograd_cannot_follow_says_so(monkeypatch, recwarn):
    """The forward functions build no graph; with a tensor that requires a gradient, in
    grad mode, they warn, once each."""
    x = torch.zeros(2, 8, requires_grad=True)
    w = {"w1": torch.zeros(16, 8), "w2": torch.zeros(8, 8)}
    p = {k: v.clone().requires_grad_() for k, v in w.items()}
    head, t = torch.zeros(5, 8), torch.zeros(2, dtype=torch.int64)
    calls = {"glu_fwd": [lambda: F.glu_fwd(x, w), lambda: F.glu_fwd(x.detach(), p),
                         lambda: F.glu_fwd(x.detach(), w, resid=x)],
             "ce_fwd": [lambda: F.ce_fwd(x, head, t),
                        lambda: F.ce_fwd(x.detach(), head.clone().requires_grad_(), t)]}
    plain = [lambda: F.glu_fwd(x.detach(), w), lambda: F.ce_fwd(x.detach(), head, t)]

    def refused():      # what follows the warning without a GPU
        return pytest.raises(ValueError, match="CUDA device")

    for name, some in calls.items():
        for call in some:
            warnings.simplefilter("always")
            monkeypatch.setattr(F, "_told", set())
            with torch.no_grad(), refused():
                call()
            assert not recwarn.list
            for _ in range(2):
                with refused():
                    call()
            assert len(recwarn.list) == 1
            assert "%s builds no autograd graph" % name in str(recwarn.pop().message)
    for call in plain:
        with refused():
            call()
    assert not recwarn.list
