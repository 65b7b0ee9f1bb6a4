"""Options of the attention functions on tensors that are not the numbers they should be, on
the CPU."""
import numpy as np
import pytest
import torch

from tensor_model_transformer_tp_gb300 import functional as F

X = torch.zeros(1, 2, 2, 8)
CALLS = [lambda **kw: F.attn_fwd(X, X, X, causal=True, **kw),
         lambda **kw: F.attn_bwd(X, X, X, X, torch.zeros(1, 2, 2), X, causal=True, **kw)]


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("name", ["q_start", "max_distance"])
@pytest.mark.parametrize("value", [1.5, 127.9, float("nan"), float("inf"), "7", "x", [3]])
def test_fractions_are_not_cut_off(call, name, value):
    with pytest.raises(ValueError, match=name):
        call(**{name: value})


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("value", [7, 7.0, np.int64(7), np.float32(7), True])
def test_whole_numbers_of_other_types(call, value):
    """(refused later, for where the tensors are)"""
    for name in ("q_start", "max_distance"):
        with pytest.raises(ValueError, match="CUDA device"):
            call(**{name: value})
    assert F._start(value) == (None, int(value)) and F._start(None) == (None, 0)
