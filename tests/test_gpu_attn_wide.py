"""Attention over keys of another length (oases_attn.h) on the GPU at sizes and starts
beside those of test_gpu_attn.py, whose definition and bounds these tests use."""
import copy

import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
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
