"""Arguments of the functions on torch tensors that no library call could carry,
refused without a GPU: shapes are given as the signatures the plans are checked
against (shape, type, CUDA device)."""
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
