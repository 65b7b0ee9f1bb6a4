"""Argument checks of oases_glu.h and oases_ce.h on the CPU: every refusal is
returned before anything is enqueued.  No kernel is launched."""
import ctypes

import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from tensor_model_transformer_tp_gb300 import functional as F

FAKE = 1 << 20  # non-NULL 16-byte aligned pointer value, never dereferenced


@pytest.fixture(scope="module", autouse=True)
def _library():
    oz.build_library()


def glu_desc(**kw):
    base = dict(dtype=1, rows=16, hidden=64, ffn=128, act=0, keep=1, dx_dtype=1, grad_dtype=0,
                accumulate=1)
    base.update(kw)
    return oz.GluDesc(*[base[n] for n, _ in oz.GluDesc._fields_])


def ce_desc(**kw):
    base = dict(ignore_index=-100, dtype=1, rows=16, hidden=64, vocab=1000, dloss_per_row=0,
                grad_dtype=0, accumulate=1)
    base.update(kw)
    return oz.CeDesc(*[base[n] for n, _ in oz.CeDesc._fields_])


def glu_status(desc, bwd=False, ws=FAKE, nb=1 << 40, **ptr):
    p = dict(w1=FAKE, b1=FAKE, w2=FAKE, b2=FAKE, x=FAKE, resid=FAKE, y=FAKE, saved=FAKE, dy=FAKE,
             dx=FAKE, gw1=FAKE, gb1=FAKE, gw2=FAKE, gb2=FAKE)
    p.update(ptr)
    w = oz.GluWeights(p["w1"], p["b1"], p["w2"], p["b2"])
    g = oz.GluGrads(p["gw1"], p["gb1"], p["gw2"], p["gb2"])
    L = oz.lib()
    if bwd:
        return L.oases_glu_bwd(ctypes.byref(desc), ctypes.byref(w), p["x"], p["dy"], p["saved"],
                               p["dx"], ctypes.byref(g), ws, nb, None)
    return L.oases_glu_fwd(ctypes.byref(desc), ctypes.byref(w), p["x"], p["resid"], p["y"],
                           p["saved"], ws, nb, None)


def ce_status(desc, bwd=False, ws=FAKE, nb=1 << 40, **ptr):
    p = dict(x=FAKE, w=FAKE, target=FAKE, loss=FAKE, lse=FAKE, dloss=FAKE, dx=FAKE, dw=FAKE)
    p.update(ptr)
    L = oz.lib()
    if bwd:
        return L.oases_ce_bwd(ctypes.byref(desc), p["x"], p["w"], p["target"], p["lse"],
                              p["dloss"], p["dx"], p["dw"], ws, nb, None)
    return L.oases_ce_fwd(ctypes.byref(desc), p["x"], p["w"], p["target"], p["loss"], p["lse"], ws,
                          nb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(dtype=-1), 1), (dict(rows=-1), 1), (dict(hidden=0), 1),
    (dict(ffn=0), 1), (dict(act=2), 1), (dict(keep=3), 1), (dict(keep=-1), 1),
    (dict(dx_dtype=2), 1), (dict(grad_dtype=2), 1), (dict(accumulate=2), 1),
    (dict(grad_dtype=1, accumulate=1), 1), (dict(dtype=0, dx_dtype=1), 1),
    (dict(hidden=60), 2), (dict(ffn=100), 2), (dict(rows=(1 << 29) + 1), 2),
    (dict(ffn=(1 << 29) + 8), 2), (dict(dtype=0, dx_dtype=0, rows=1 << 22), 2), (dict(dtype=0, dx_dtype=0, keep=2), 2),
])
def test_glu_descriptors(bad, status):
    d = glu_desc(**bad)
    assert glu_status(d) == status and glu_status(d, bwd=True) == status
    assert oz.oases_glu_workspace_bytes(d, False) == oz.oases_glu_workspace_bytes(d, True) == 0
    assert oz.oases_glu_saved_bytes(d) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(rows=-1), 1), (dict(hidden=0), 1), (dict(vocab=0), 1),
    (dict(dloss_per_row=2), 1), (dict(grad_dtype=2), 1), (dict(accumulate=-1), 1),
    (dict(grad_dtype=1, accumulate=1), 1), (dict(hidden=36), 2), (dict(vocab=(1 << 29) + 1), 2),
    (dict(dtype=0, vocab=1 << 22), 2),
])
def test_ce_descriptors(bad, status):
    d = ce_desc(**bad)
    assert ce_status(d) == status and ce_status(d, bwd=True) == status
    assert oz.oases_ce_workspace_bytes(d, False) == oz.oases_ce_workspace_bytes(d, True) == 0


def test_pointers_and_workspaces():
    d = glu_desc()
    for name in ("x", "w1", "w2", "y", "saved"):
        assert glu_status(d, **{name: None}) == 1
    for name in ("x", "w1", "b1", "w2", "b2", "resid", "y", "saved"):
        assert glu_status(d, **{name: FAKE + 8}) == 1
    for name in ("x", "w1", "w2", "dy", "saved"):
        assert glu_status(d, bwd=True, **{name: None}) == 1
    for name in ("x", "dy", "dx", "gw1", "gb1", "gw2", "gb2"):
        assert glu_status(d, bwd=True, **{name: FAKE + 4}) == 1
    assert glu_status(d, bwd=True, b1=None) == 1      # a gradient of a bias that is not there
    c = ce_desc()
    for name in ("x", "w", "target", "loss", "lse"):
        assert ce_status(c, **{name: None}) == 1
    for name, off in (("x", 8), ("w", 8), ("target", 4), ("loss", 2), ("lse", 2)):
        assert ce_status(c, **{name: FAKE + off}) == 1
    for name in ("x", "w", "target", "lse", "dloss"):
        assert ce_status(c, bwd=True, **{name: None}) == 1
    for name, off in (("dx", 8), ("dw", 8), ("target", 4), ("lse", 2), ("dloss", 2)):
        assert ce_status(c, bwd=True, **{name: FAKE + off}) == 1
    for bwd in (False, True):
        for need, status, desc in ((oz.oases_glu_workspace_bytes(d, bwd), glu_status, d),
                                   (oz.oases_ce_workspace_bytes(c, bwd), ce_status, c)):
            if need:
                assert status(desc, bwd, ws=None) == 3
                assert status(desc, bwd, nb=need - 1) == 3


def test_workspaces_of_every_size_can_be_asked_for():
    """From one row to millions, without a device: positive, and no smaller for
    more rows than what the rows' own intermediate results need."""
    for rows in (1, 127, 128, 129, 256, 1000, 8192, 100000, 1 << 22):
        for keep in (0, 1, 2):
            d = glu_desc(rows=rows, hidden=2560, ffn=10240, keep=keep)
            assert oz.oases_glu_workspace_bytes(d, False) >= rows * 10240 * 2
            assert oz.oases_glu_workspace_bytes(d, True) >= rows * 3 * 10240 * 2
        c = ce_desc(rows=rows, hidden=2560, vocab=50257)
        assert oz.oases_ce_workspace_bytes(c, False) > 0
        # g of one piece, not of the whole vocabulary
        n = oz.oases_ce_workspace_bytes(c, True)
        assert 0 < n <= (600 << 20) + rows * (4096 + 256) * 2 + rows * 2560 * 4


def test_no_rows_need_nothing():
    d, c = glu_desc(rows=0), ce_desc(rows=0)
    assert glu_status(d, ws=None, nb=0, x=None, y=None, saved=None) == 0
    assert glu_status(d, bwd=True, ws=None, nb=0, x=None, dy=None, saved=None, dx=None) == 0
    assert ce_status(c, ws=None, nb=0, x=None, target=None, loss=None, lse=None) == 0
    assert ce_status(c, bwd=True, ws=None, nb=0, x=None, lse=None, dloss=None, dx=None) == 0


def test_saved_bytes():
    assert oz.oases_glu_saved_bytes(glu_desc(keep=0)) == 0
    assert oz.oases_glu_saved_bytes(glu_desc(keep=1)) == 16 * 256 * 2
    assert oz.oases_glu_saved_bytes(glu_desc(keep=1, dtype=0, dx_dtype=0)) == 16 * 256 * 4
    # codes 2 * 16 * 128, scales one 512-byte tile per projection
    assert oz.oases_glu_saved_bytes(glu_desc(keep=2)) == 4096 + 1024
    assert oz.oases_glu_saved_bytes(glu_desc(keep=2, rows=130, ffn=136)) == \
        (2 * 130 * 144 + 255) // 256 * 256 + 2 * 2 * 2 * 512


def test_functions_on_tensors_refuse_the_cpu():
    x = torch.zeros(2, 8)
    w = {"w1": torch.zeros(16, 8), "w2": torch.zeros(8, 8)}
    with pytest.raises(ValueError):
        F.glu_fwd(x, w)
    with pytest.raises(ValueError):
        F.glu_bwd(x, x, w)
    with pytest.raises(ValueError):
        F.ce_fwd(x, torch.zeros(5, 8), torch.zeros(2, dtype=torch.int64))
