"""Argument checks of oases_attn.h and oases_qknorm.h, and of the functions on tensors
above them, on the CPU: every refusal is returned before anything is enqueued.  No
kernel is launched."""
import ctypes

import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from tensor_model_transformer_tp_gb300 import functional as F

FAKE = 1 << 20  # non-NULL 16-byte aligned pointer value, never dereferenced
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _library():
    oz.build_library()


def attn_desc(**kw):
    base = dict(dtype=1, batch=2, q_len=5, k_len=70, heads=4, kv_heads=2, head_dim=64, causal=0,
                q_start=0, buckets=32, max_distance=128, bidirectional=1, grad_dtype=0,
                accumulate=1, scale=0.125)
    strides = {n: oz.Strides(5 * 256, 256, 64) for n in ("q", "o", "d_o", "dq")}
    strides |= {n: oz.Strides(70 * 128, 128, 64) for n in ("k", "v", "dk", "dv")}
    return oz.AttnDesc(**(base | strides | kw))


def attn_status(desc, bwd=False, ws=FAKE, nb=1 << 40, **ptr):
    p = {n: FAKE for n in ("q", "k", "v", "kv_lens", "q_start", "bias", "o", "lse", "d_o", "dq",
                           "dk", "dv", "dbias")} | ptr
    names = ["q", "k", "v", "kv_lens", "q_start", "bias", "o", "lse"]
    names += ["d_o", "dq", "dk", "dv", "dbias"] if bwd else []
    fn = oz.lib().oases_attn_bwd if bwd else oz.lib().oases_attn_fwd
    return fn(ctypes.byref(desc), *[p[n] for n in names], ws, nb, None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(batch=-1), 1), (dict(q_len=-1), 1), (dict(k_len=-1), 1),
    (dict(heads=0), 1), (dict(kv_heads=0), 1), (dict(kv_heads=3), 1), (dict(head_dim=0), 1),
    (dict(causal=2), 1), (dict(q_start=-1), 1), (dict(buckets=1), 1), (dict(buckets=-4), 1),
    (dict(buckets=2), 1), (dict(buckets=33), 1), (dict(max_distance=8), 1),
    (dict(bidirectional=0, max_distance=16), 1), (dict(bidirectional=2), 1),
    (dict(grad_dtype=1), 1), (dict(grad_dtype=2), 1), (dict(accumulate=2), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1),
    (dict(scale=float("nan")), 1), (dict(q=oz.Strides(1280, 252, 64)), 1),
    (dict(k=oz.Strides(0, 128, 64)), 1), (dict(v=oz.Strides(8960, 128, -64)), 1),
    (dict(o=oz.Strides(1280, 256, (1 << 36) + 8)), 1),
    (dict(head_dim=60), 2), (dict(head_dim=136), 2), (dict(buckets=130), 2),
    (dict(max_distance=65537), 2), (dict(k_len=(1 << 24) + 1), 2), (dict(batch=1 << 23), 2),
])
def test_attention_descriptors(bad, status):
    d = attn_desc(**bad)
    assert attn_status(d) == status and attn_status(d, bwd=True) == status
    assert oz.oases_attn_workspace_bytes(d, False) == oz.oases_attn_workspace_bytes(d, True) == 0


def test_strides_of_one_element_are_not_read():
    d = attn_desc(batch=1, kv_heads=1, heads=1, q=oz.Strides(-3, 64, 1), k=oz.Strides(0, 64, 0))
    assert oz.oases_attn_workspace_bytes(d, True) > 0
    assert attn_status(attn_desc(dq=oz.Strides(3, 256, 64)), bwd=True) == 1
    assert attn_status(attn_desc(dq=oz.Strides(3, 256, 64)), ws=None) == 3


def test_attention_pointers_and_workspaces():
    d = attn_desc()
    for name in ("q", "k", "v", "bias", "o", "lse"):
        assert attn_status(d, **{name: None}) == 1
        assert attn_status(d, bwd=True, **{name: None}) == 1
    for name in ("d_o", "dq", "dk", "dv"):
        assert attn_status(d, bwd=True, **{name: None}) == 1
        assert attn_status(d, bwd=True, **{name: FAKE + 8}) == 1
    for name, off in (("q", 8), ("k", 8), ("v", 8), ("o", 8), ("lse", 2), ("kv_lens", 2),
                      ("q_start", 2), ("bias", 1)):
        assert attn_status(d, **{name: FAKE + off}) == 1
    assert attn_status(d, bwd=True, dbias=FAKE + 2) == 1
    plain = attn_desc(buckets=0)
    assert attn_status(plain) == 1                               # a bias that has no buckets
    assert attn_status(plain, bwd=True, bias=None) == 1          # a gradient of none
    for bwd in (False, True):
        need = oz.oases_attn_workspace_bytes(d, bwd)
        assert need > 0
        assert attn_status(d, bwd, ws=None) == 3 and attn_status(d, bwd, nb=need - 1) == 3
        assert attn_status(d, bwd, ws=FAKE + 8) == 1


def test_nothing_to_do_needs_nothing():
    for d in (attn_desc(batch=0), attn_desc(q_len=0)):
        assert attn_status(d, ws=None, nb=0, q=None, o=None, lse=None) == 0


def qk_desc(**kw):
    base = dict(dtype=1, batch=2, seq=9, heads=4, kv_heads=2, head_dim=64, rot=32, interleaved=0,
                positions_len=50, positions_shared=0, grad_dtype=0, accumulate=1, eps=1e-6)
    strides = {n: oz.Strides(9 * 256, 256, 64) for n in ("q", "q_out", "dq")}
    strides |= {n: oz.Strides(9 * 128, 128, 64) for n in ("k", "k_out", "dk")}
    return oz.QknormDesc(**(base | strides | kw))


def qk_status(desc, bwd=False, ws=FAKE, nb=1 << 40, **ptr):
    p = {n: FAKE for n in ("q", "k", "dqo", "dko", "cos", "sin", "positions", "wq", "wk", "qo",
                           "ko", "dq", "dk", "dwq", "dwk")} | ptr
    L = oz.lib()
    if bwd:
        return L.oases_qknorm_bwd(ctypes.byref(desc), *[p[n] for n in (
            "q", "k", "dqo", "dko", "cos", "sin", "positions", "wq", "wk", "dq", "dk", "dwq",
            "dwk")], ws, nb, None)
    return L.oases_qknorm_fwd(ctypes.byref(desc), *[p[n] for n in (
        "q", "k", "cos", "sin", "positions", "wq", "wk", "qo", "ko")], None)


@pytest.mark.parametrize("bad,status", [
    (dict(dtype=2), 1), (dict(batch=-1), 1), (dict(seq=-1), 1), (dict(heads=-1), 1),
    (dict(kv_heads=-1), 1), (dict(head_dim=0), 1), (dict(rot=33), 1), (dict(rot=66), 1),
    (dict(rot=-2), 1), (dict(interleaved=2), 1), (dict(positions_len=-1), 1),
    (dict(positions_shared=2), 1), (dict(grad_dtype=1), 1), (dict(eps=0.0), 1),
    (dict(eps=float("nan")), 1), (dict(q=oz.Strides(2304, 260, 64)), 1),
    (dict(k_out=oz.Strides(1152, -128, 64)), 1), (dict(head_dim=60, rot=0), 2),
    (dict(head_dim=264), 2), (dict(batch=1 << 28, seq=9), 2),
])
def test_norm_descriptors(bad, status):
    d = qk_desc(**bad)
    assert qk_status(d) == status and qk_status(d, bwd=True) == status
    assert oz.oases_qknorm_workspace_bytes(d) == 0


def test_norm_pointers():
    d = qk_desc()
    for name in ("q", "k", "cos", "sin", "qo", "ko"):
        assert qk_status(d, **{name: None}) == 1
    for name, off in (("q", 8), ("k", 8), ("qo", 8), ("ko", 8), ("wq", 8), ("cos", 2),
                      ("positions", 4)):
        assert qk_status(d, **{name: FAKE + off}) == 1
    for name in ("q", "k", "dqo", "dko", "cos", "sin"):
        assert qk_status(d, bwd=True, **{name: None}) == 1
    assert qk_status(d, bwd=True, wq=None) == 1      # a gradient of a weight that is not there
    need = oz.oases_qknorm_workspace_bytes(d)
    assert need > 0 and qk_status(d, True, ws=None) == 3 and qk_status(d, True, nb=need - 1) == 3
    none = qk_desc(seq=0)
    assert qk_status(none, q=None, qo=None) == 0
    assert qk_status(none, bwd=True, ws=None, nb=0, q=None, dqo=None) == 0


# ---- the functions on tensors: shapes given as the views their plans are checked against ----
def view(*shape, dtype=BF, stride=None):
    return torch.Size(shape), stride or torch.empty(shape, device="meta").stride(), dtype, 0


def sig(*shape, dtype=BF):
    return torch.Size(shape), dtype, 0


OPT = (False, 0, None, 128, True)


@pytest.fixture(autouse=True)
def _plans_without_a_device(monkeypatch):
    """Plans that pass ask the library for sizes on the tensors' device: not here."""
    monkeypatch.setattr(F, "_sized", lambda index, *asked: tuple(0 for _ in asked))
    yield
    for plan in (F._attn_fwd_plan, F._attn_bwd_plan, F._qknorm_bwd_plan):
        plan.cache_clear()


def fwd_plan(q=view(2, 5, 4, 64), k=view(2, 9, 2, 64), v=view(2, 9, 2, 64), lens=None, start=None,
             bias=None, opt=OPT):
    return F._attn_fwd_plan(q, k, v, lens, start, bias, *opt)


@pytest.mark.parametrize("bad,match", [
    (dict(q=view(5, 4, 64)), "q must be"), (dict(q=view(2, 5, 4, 64, dtype=torch.float16)), "q must"),
    (dict(k=view(2, 9, 3, 64), v=view(2, 9, 3, 64)), "do not share"), (dict(v=view(2, 8, 2, 64)), "v must"),
    (dict(k=view(3, 9, 2, 64)), "k must"), (dict(k=view(2, 9, 2, 32)), "k must"),
    (dict(k=view(2, 9, 2, 64, dtype=torch.float32)), "k must"),
    (dict(q=view(2, 5, 4, 64, stride=(1280, 256, 1, 4))), "side by side"),
    (dict(k=view(2, 9, 2, 64, stride=(0, 128, 64, 1))), "k's strides"),
    (dict(v=view(2, 9, 2, 64, stride=(1170, 130, 64, 1))), "v's strides"),
    (dict(lens=sig(2)), "kv_lens"), (dict(lens=sig(3, dtype=torch.int32)), "kv_lens"),
    (dict(start=sig(2, dtype=torch.int64)), "q_start"), (dict(opt=(True, -1, None, 128, True)), "q_start"),
    (dict(opt=(True, 1 << 31, None, 128, True)), "q_start"),
    (dict(bias=sig(32, 3)), "bias"), (dict(bias=sig(32, 4, dtype=torch.float32)), "bias"),
    (dict(bias=sig(32, 4), opt=(False, 0, None, 1 << 40, True)), "max_distance"),
    (dict(q=view(1 << 32, 5, 4, 64)), "dimension 0"),
])
def test_attention_tensors(bad, match):
    fwd_plan()
    with pytest.raises(ValueError, match=match):
        fwd_plan(**bad)


def test_attention_backward_tensors():
    q, k = view(2, 5, 4, 64), view(2, 9, 2, 64)
    good = dict(o=q, lse=sig(2, 4, 5, dtype=torch.float32), do=q, outs=(None, None, None), bias=None,
                dbias=None, need=True)

    def plan(**kw):
        a = good | kw
        return F._attn_bwd_plan(q, k, k, a["o"], a["lse"], a["do"], a["outs"], None, None, a["bias"],
                                a["dbias"], a["need"], *OPT)

    plan()
    f32 = torch.float32
    for bad, match in ((dict(o=k), "o must"), (dict(do=None), "do must"), (dict(lse=sig(2, 4, 5)), "lse"),
                       (dict(outs=(None, q, None)), "dk must"),
                       (dict(dbias=sig(32, 4, dtype=f32)), "dbias is given"),
                       (dict(bias=sig(32, 4), dbias=sig(32, 4)), "dbias must"),
                       (dict(bias=sig(32, 4), dbias=sig(32, 4, dtype=f32), need=False), "dbias is given")):
        with pytest.raises(ValueError, match=match):
            plan(**bad)


def test_norm_tensors():
    q, k, f32 = view(2, 9, 4, 64), view(2, 9, 2, 64), torch.float32
    good = dict(k=k, outs=(None, None), cos=sig(50, 16, dtype=f32), sin=sig(50, 16, dtype=f32),
                positions=None, wq=None, wk=None)

    def plan(**kw):
        a = good | kw
        return F._qknorm_fwd_plan(q, a["k"], a["outs"], a["cos"], a["sin"], a["positions"], a["wq"],
                                  a["wk"], 1e-6, False)

    plan()
    for bad, match in ((dict(k=view(2, 8, 2, 64)), "k must"), (dict(wq=sig(32)), "q_weight"),
                       (dict(k=None, wk=sig(64)), "no k"), (dict(sin=None), "belong together"),
                       (dict(cos=sig(50, 16)), "cos must"), (dict(sin=sig(50, 8, dtype=f32)), "sin must"),
                       (dict(cos=sig(50, 33, dtype=f32), sin=sig(50, 33, dtype=f32)), "66 values"),
                       (dict(cos=sig(5, 16, dtype=f32), sin=sig(5, 16, dtype=f32)), "hold 5 positions"),
                       (dict(positions=sig(2, 9, dtype=torch.int32)), "positions"),
                       (dict(positions=sig(3, 9, dtype=torch.int64)), "positions"),
                       (dict(cos=None, sin=None, positions=sig(2, 9, dtype=torch.int64)), "no tables"),
                       (dict(k=None, outs=(None, q)), "no k"), (dict(outs=(k, None)), "q_out must")):
        with pytest.raises(ValueError, match=match):
            plan(**bad)


def test_tensors_on_the_cpu_are_refused():
    x = torch.zeros(1, 2, 2, 8)
    with pytest.raises(ValueError, match="CUDA device"):
        F.attn_fwd(x, x, x)
    with pytest.raises(ValueError, match="CUDA device"):
        F.attn_bwd(x, x, x, x, torch.zeros(1, 2, 2), x)
    with pytest.raises(ValueError, match="CUDA device"):
        F.qk_norm_rope_fwd(x, x, None, None)
    with pytest.raises(ValueError, match="CUDA device"):
        F.qk_norm_rope_bwd(x, x, x, x, None, None)
