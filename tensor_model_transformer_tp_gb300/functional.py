"""The gated feed-forward block, the linear head's cross entropy, attention over keys
of another length and the norms and rotation in front of it, on torch tensors.

Each function checks its tensors (once per combination of shapes, types and
options), allocates outputs and workspace with torch's caching allocator and makes
one call of liboases.so on torch's current stream of the tensors' device; nothing
is computed here and no data is kept between calls.  Because the allocations
follow torch's stream rules, the calls can be made on any stream, from several
threads, and inside CUDA graph capture.

Tensors are contiguous, on one CUDA device, ``float32`` or ``bfloat16`` as
``x`` is; anything else raises ``ValueError`` before a call is made.  (The
four-dimensional tensors of the attention functions need only a head's values side
by side and strides of whole 16 bytes: slices of a packed projection are taken as
they are.)  Errors of the library raise ``OasesError``.  There is no autograd integration: the
backward functions are called with what the forward returned.  (A forward function
given a tensor that requires a gradient, in grad mode, warns of it once.)
"""
from __future__ import annotations

import ctypes
import functools
import warnings
from typing import Dict, Optional, Tuple, Union

import torch

from . import (ACT, KEEP, AttnDesc, CeDesc, GluDesc, GluGrads, GluWeights, QknormDesc, Strides,
               _check as _check_status, lib, oases_attn_workspace_bytes, oases_ce_workspace_bytes,
               oases_glu_saved_bytes, oases_glu_workspace_bytes, oases_qknorm_workspace_bytes)

_CODE = {torch.float32: 0, torch.bfloat16: 1}
_NAMES = ("w1", "b1", "w2", "b2")
_get_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_raw_alloc = torch._C._cuda_cudaCachingAllocator_raw_alloc
_raw_delete = torch._C._cuda_cudaCachingAllocator_raw_delete


_told = set()


def _no_graph(name: str, *tensors: Optional[torch.Tensor]) -> None:
    """Warn, once a function, where autograd would have followed the call."""
    if name in _told or not torch.is_grad_enabled():
        return
    for t in tensors:
        if t is not None and t.requires_grad:
            _told.add(name)
            warnings.warn("%s builds no autograd graph: call the backward function for the "
                          "gradients, or wrap both in a torch.autograd.Function" % name,
                          stacklevel=3)
            return


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _sig(t: Optional[torch.Tensor]):
    """What a plan is checked against: shape, type and CUDA device (-1 for the
    CPU); None where there is no tensor."""
    if t is None:
        return None
    try:
        if t.is_contiguous():
            return t.shape, t.dtype, t.get_device()
    except AttributeError:
        raise ValueError("expected a tensor or None, got %s" % type(t)) from None
    raise ValueError("a tensor of shape %s is not contiguous" % (tuple(t.shape),))


def _match(name: str, sig, shape: tuple, dtype: torch.dtype, device) -> None:
    if sig is None or tuple(sig[0]) != shape or sig[1] != dtype:
        raise ValueError("%s must be a %s tensor of shape %s, got %s" % (
            name, dtype, shape, None if sig is None else (sig[1], tuple(sig[0]))))
    if sig[2] != device:
        raise ValueError("%s is on device %d, x on %d" % (name, sig[2], device))


def _fits(**sizes: int) -> None:
    """The descriptors hold 32-bit sizes, which ctypes would cut off in silence."""
    for name, n in sizes.items():
        _need(n < 1 << 31, "%s is %d, beyond 2^31 - 1" % (name, n))


def _rows(x) -> Tuple[int, int]:
    _need(x is not None and len(x[0]) == 2, "x must be a [rows, hidden] tensor")
    _need(x[1] in _CODE, "x must be float32 or bfloat16, got %s" % (x[1],))
    _need(x[2] >= 0, "x must be on a CUDA device")
    _fits(rows=x[0][0], hidden=x[0][1])
    return x[0][0], x[0][1]


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _call(fn, index: int, n_ws: int, *args) -> None:
    """One library call on torch's current stream of device ``index``, made
    current, with n_ws bytes of workspace from torch's caching allocator (raw, as
    torch.cuda.caching_allocator_alloc gives it: a third of a tensor's cost)."""
    if _get_device() != index:
        with torch.cuda.device(index):
            return _call(fn, index, n_ws, *args)
    stream = _raw_stream(index)
    if n_ws:
        ws = _raw_alloc(n_ws, stream)
        try:
            st = fn(*args, ws, n_ws, stream)
        finally:
            _raw_delete(ws)
    else:
        st = fn(*args, None, 0, stream)
    if st:
        _check_status(st)


def _call_no_ws(fn, index: int, *args) -> None:
    """_call for a function that takes no workspace."""
    if _get_device() != index:
        with torch.cuda.device(index):
            return _call_no_ws(fn, index, *args)
    st = fn(*args, _raw_stream(index))
    if st:
        _check_status(st)


def _sized(index: int, *asked):
    """The library's answers about sizes, for the device (its number of SMs)."""
    with torch.cuda.device(index):
        return tuple(f(*a) for f, *a in asked)


# ---- gated feed-forward block ---------------------------------------------------
# Plans are checked once per combination of shapes, types and options.
def _glu_shapes(x, w):
    rows, hidden = _rows(x)
    _need(w[0] is not None and w[2] is not None, "weights needs w1 and w2")
    _need(len(w[2][0]) == 2, "w2 must be [hidden, ffn]")
    ffn = w[2][0][1]
    _fits(ffn=ffn)
    shapes = {"w1": (2 * ffn, hidden), "b1": (2 * ffn,), "w2": (hidden, ffn), "b2": (hidden,)}
    for name, sig in zip(_NAMES, w):
        if sig is not None:
            _match(name, sig, shapes[name], x[1], x[2])
    return rows, hidden, ffn, shapes


def _glu_options(act, save):
    _need(act in ACT, "act must be one of %s" % sorted(ACT))
    _need(save in KEEP, "save must be one of %s" % sorted(KEEP))


@functools.lru_cache(maxsize=512)
def _glu_fwd_plan(x, w, resid, y, act, save):
    rows, hidden, ffn, _ = _glu_shapes(x, w)
    _glu_options(act, save)
    for name, sig in (("resid", resid), ("y", y)):
        if sig is not None:
            _match(name, sig, (rows, hidden), x[1], x[2])
    t = _CODE[x[1]]
    d = GluDesc(t, rows, hidden, ffn, ACT[act], KEEP[save], t, t, 0)
    return (ctypes.byref(d), oases_glu_saved_bytes(d),
            *_sized(x[2], (oases_glu_workspace_bytes, d, False)), (rows, 2 * ffn))


@functools.lru_cache(maxsize=512)
def _glu_bwd_plan(x, w, dy, saved, grads, act, save, dx_dtype):
    rows, hidden, ffn, shapes = _glu_shapes(x, w)
    _glu_options(act, save)
    _match("dy", dy, (rows, hidden), x[1], x[2])
    accumulate = grads is not None
    if accumulate:
        for name, sig, weight in zip(_NAMES, grads, w):
            if sig is not None:
                _need(weight is not None, "grads[%r] has no weight" % name)
                _match("grads[%r]" % name, sig, shapes[name], torch.float32, x[2])
    _need(dx_dtype in (None, x[1], torch.float32), "dx_dtype must be x's type or float32")
    t = _CODE[x[1]]
    d = GluDesc(t, rows, hidden, ffn, ACT[act], KEEP[save], t if dx_dtype is None else
                _CODE[dx_dtype], 0 if accumulate else t, int(accumulate))
    if save == "none":
        _need(saved is None, "saved is given, but save is \"none\"")
    elif save == "pre":
        _match("saved", saved, (rows, 2 * ffn), x[1], x[2])
    else:
        _match("saved", saved, (oases_glu_saved_bytes(d),), torch.uint8, x[2])
    return (ctypes.byref(d), *_sized(x[2], (oases_glu_workspace_bytes, d, True)))


def _named(tensors: Dict[str, torch.Tensor], what: str):
    if not tensors.keys() <= set(_NAMES):
        raise ValueError("unknown %s %s" % (what, sorted(set(tensors) - set(_NAMES))))
    get = tensors.get
    return get("w1"), get("b1"), get("w2"), get("b2")


def glu_fwd(x: torch.Tensor, weights: Dict[str, torch.Tensor], act: str = "silu",
            resid: Optional[torch.Tensor] = None, save: str = "none",
            y: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """y = (act(x Wg^T + bg) * (x Wu^T + bu)) W2^T + b2 (+ resid).

    x [rows, hidden]; weights: "w1" [2 ffn, hidden] = [Wg; Wu], "w2"
    [hidden, ffn] and optionally "b1" [2 ffn], "b2" [hidden].  act: "silu" or
    "gelu" (exact).  save: what is kept for the backward beside x: "none",
    "pre" ([a | b], [rows, 2 ffn] in x's type) or "mxfp8" (a and b in 8 bits, a
    byte tensor in the layout of oases_glu.h; bfloat16 only).  "none" is the most
    accurate in bfloat16: the backward forms a and b in fp32 again, where "pre" has
    them rounded (gradients 0.0035 of their size off against 0.0024).
    Returns (y, kept activations or None).  y may be given (resid itself, for
    an in-place residual).
    """
    w1, b1, w2, b2 = _named(weights, "weights")
    sigs = _sig(x), (_sig(w1), _sig(b1), _sig(w2), _sig(b2)), _sig(resid), _sig(y)
    _no_graph("glu_fwd", x, w1, b1, w2, b2, resid)
    desc, n_saved, n_ws, kept = _glu_fwd_plan(*sigs, act, save)
    if y is None:
        y = torch.empty_like(x)
    saved = None
    if save == "pre":
        saved = torch.empty(kept, dtype=x.dtype, device=x.device)
    elif save == "mxfp8":
        saved = torch.empty(n_saved, dtype=torch.uint8, device=x.device)
    w = GluWeights(_ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2))
    _call(lib().oases_glu_fwd, x.get_device(), n_ws, desc, ctypes.byref(w), _ptr(x), _ptr(resid),
          _ptr(y), _ptr(saved))
    return y, saved


def glu_bwd(x: torch.Tensor, dy: torch.Tensor, weights: Dict[str, torch.Tensor],
            act: str = "silu", save: str = "none", saved: Optional[torch.Tensor] = None,
            grads: Optional[Dict[str, torch.Tensor]] = None,
            dx_dtype: Optional[torch.dtype] = None, need_dx: bool = True
            ) -> Tuple[Optional[torch.Tensor], Dict[str, torch.Tensor]]:
    """Backward of glu_fwd for the output gradient dy, with the same x, weights,
    act and save, and the activations it kept.

    grads None: the gradients of every weight given are returned in x's type.
    grads a dict of float32 tensors (any subset of the weights' names): they are
    added to (+=), the convention of the block; the rest are left out.
    dx_dtype: x's type (default) or float32.  Returns (dx or None, grads).
    """
    w1, b1, w2, b2 = _named(weights, "weights")
    given = None if grads is None else _named(grads, "grads")
    desc, n_ws = _glu_bwd_plan(
        _sig(x), (_sig(w1), _sig(b1), _sig(w2), _sig(b2)), _sig(dy), _sig(saved),
        None if given is None else tuple(_sig(g) for g in given), act, save, dx_dtype)
    if grads is None:
        grads = {k: torch.empty_like(v) for k, v in weights.items() if v is not None}
        given = _named(grads, "grads")
    dx = torch.empty_like(x, dtype=dx_dtype) if need_dx else None
    w = GluWeights(_ptr(w1), _ptr(b1), _ptr(w2), _ptr(b2))
    g = GluGrads(*[_ptr(v) for v in given])
    _call(lib().oases_glu_bwd, x.get_device(), n_ws, desc, ctypes.byref(w), _ptr(x), _ptr(dy),
          _ptr(saved), _ptr(dx), ctypes.byref(g))
    return dx, grads


# ---- cross entropy of the linear head -----------------------------------------------
@functools.lru_cache(maxsize=512)
def _ce_plan(x, w, targets, lse, dloss, dw, backward, ignore_index):
    rows, hidden = _rows(x)
    _need(w is not None and len(w[0]) == 2 and w[0][0] > 0, "w must be a [vocab, hidden] tensor")
    vocab = w[0][0]
    _fits(vocab=vocab)
    _need(-1 << 63 <= ignore_index < 1 << 63, "ignore_index must be a 64-bit integer")
    _match("w", w, (vocab, hidden), x[1], x[2])
    _match("targets", targets, (rows,), torch.int64, x[2])
    t, per_row, accumulate = _CODE[x[1]], False, dw is not None
    if backward:
        _match("lse", lse, (rows,), torch.float32, x[2])
        _need(dloss is not None, "dloss must be a tensor")
        per_row = tuple(dloss[0]) not in ((), (1,))
        _match("dloss", dloss, (rows,) if per_row else tuple(dloss[0]), torch.float32, x[2])
    if accumulate:
        _match("dw", dw, (vocab, hidden), torch.float32, x[2])
    d = CeDesc(ignore_index, t, rows, hidden, vocab, int(per_row), 0 if accumulate else t,
               int(accumulate))
    return (ctypes.byref(d), *_sized(x[2], (oases_ce_workspace_bytes, d, backward)), rows)


def ce_fwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
           ignore_index: int = -100) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-row cross entropy of the logits x w^T: (loss, lse), float32 [rows].

    x [rows, hidden], w [vocab, hidden], targets int64 [rows].  Rows whose
    target is ignore_index have loss 0; another target outside [0, vocab)
    gives NaN.  The logits are not kept.
    """
    sigs = _sig(x), _sig(w), _sig(targets)
    _no_graph("ce_fwd", x, w)
    desc, n_ws, rows = _ce_plan(*sigs, None, None, None, False, ignore_index)
    loss = torch.empty(rows, dtype=torch.float32, device=x.device)
    lse = torch.empty_like(loss)
    _call(lib().oases_ce_fwd, x.get_device(), n_ws, desc, _ptr(x), _ptr(w), _ptr(targets), _ptr(loss),
          _ptr(lse))
    return loss, lse


def ce_bwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
           dloss: torch.Tensor, dw: Optional[torch.Tensor] = None, ignore_index: int = -100,
           need_dx: bool = True, need_dw: bool = True
           ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients (dx, dw) of ce_fwd for the gradient dloss of its losses:
    float32, [rows], or [1] (or a scalar tensor) for the same value in every row
    (1 / n for the mean over n rows with a loss).

    In bfloat16 the gradient of the logits is rounded to bfloat16, the operand type
    of dx and dw, after a common factor of the rows has been taken out; dtype
    float32 rounds nothing but fp32 sums.
    dw None: returned in x's type.  dw a float32 [vocab, hidden] tensor: it is
    added to (+=) and returned.  Ignored rows of x count in dw times 0: they must
    be finite.
    """
    desc, n_ws, _ = _ce_plan(_sig(x), _sig(w), _sig(targets), _sig(lse), _sig(dloss), _sig(dw),
                             True, ignore_index)
    _need(need_dw or dw is None, "dw is given, but need_dw is false")
    if dw is None and need_dw:
        dw = torch.empty_like(w)
    dx = torch.empty_like(x) if need_dx else None
    _call(lib().oases_ce_bwd, x.get_device(), n_ws, desc, _ptr(x), _ptr(w), _ptr(targets), _ptr(lse),
          _ptr(dloss), _ptr(dx), _ptr(dw))
    return dx, dw


# ---- attention over keys of another length --------------------------------------------
def _view(t: Optional[torch.Tensor]):
    """As _sig, of a tensor whose strides are its own: shape, strides, type, device."""
    if t is None:
        return None
    try:
        return t.shape, t.stride(), t.dtype, t.get_device()
    except AttributeError:
        raise ValueError("expected a tensor or None, got %s" % type(t)) from None


def _heads_of(name: str, v, like=None) -> Strides:
    """The strides of a [batch, tokens, heads, head_dim] view (of shape, type and device
    `like`, where given)."""
    _need(v is not None and len(v[0]) == 4,
          "%s must be a [batch, tokens, heads, head_dim] tensor" % name)
    shape, stride, dtype, device = v
    if like is not None:
        want, dt, dev = like
        if tuple(shape) != want or dtype != dt:
            raise ValueError("%s must be a %s tensor of shape %s, got %s" % (
                name, dt, want, (dtype, tuple(shape))))
        _need(device == dev, "%s is on device %d, q on %d" % (name, device, dev))
    _need(dtype in _CODE, "%s must be float32 or bfloat16, got %s" % (name, dtype))
    _need(device >= 0, "%s must be on a CUDA device" % name)
    _fits(**{"%s's dimension %d" % (name, i): n for i, n in enumerate(shape)})
    _need(shape[3] <= 1 or stride[3] == 1, "%s's head values must be side by side" % name)
    per = 16 // dtype.itemsize
    for n, s in zip(shape[:3], stride[:3]):
        _need(n <= 1 or (s > 0 and s % per == 0),
              "%s's strides %s are not all positive multiples of 16 bytes" % (name, tuple(stride)))
    return Strides(*stride[:3])


def _like(v):
    return tuple(v[0]), v[2], v[3]


def _attn_common(q, k, v, kv_lens, q_start, bias, causal, start, scale, max_distance,
                 bidirectional):
    """The descriptor's fields that both directions share."""
    sq, sk = _heads_of("q", q), _heads_of("k", k)
    (B, Sq, H, D), dtype, dev = _like(q)
    Sk, G = k[0][1], k[0][2]
    _heads_of("k", k, ((B, Sk, G, D), dtype, dev))
    sv = _heads_of("v", v, ((B, Sk, G, D), dtype, dev))
    _need(H > 0 and G > 0 and H % G == 0, "%d query heads do not share %d key heads" % (H, G))
    for name, t in (("kv_lens", kv_lens), ("q_start", q_start)):
        if t is not None:
            _match(name, t, (B,), torch.int32, dev)
    _need(0 <= start < 1 << 31, "q_start is %d, negative or beyond 2^31 - 1" % start)
    buckets = 0
    if bias is not None:
        _need(len(bias[0]) == 2, "bias must be [buckets, heads]")
        buckets = bias[0][0]
        _match("bias", bias, (buckets, H), dtype, dev)
        _need(2 <= buckets < 1 << 31, "bias has %d buckets" % buckets)
        _need(0 < max_distance < 1 << 31, "max_distance is %d" % max_distance)
    return dict(dtype=_CODE[dtype], batch=B, q_len=Sq, k_len=Sk, heads=H, kv_heads=G, head_dim=D,
                causal=int(causal), q_start=start, buckets=buckets, max_distance=max_distance,
                bidirectional=int(bidirectional),
                scale=D ** -0.5 if scale is None else scale, q=sq, k=sk, v=sv)


_NO_OUT = (None, None, None)


def _row_strides(shape) -> Strides:
    """Of a contiguous [batch, tokens, heads, head_dim] tensor."""
    B, S, H, D = shape
    return Strides(S * H * D, H * D, D)


@functools.lru_cache(maxsize=512)
def _attn_fwd_plan(q, k, v, kv_lens, q_start, bias, *options):
    d = AttnDesc(**_attn_common(q, k, v, kv_lens, q_start, bias, *options))
    d.o = _row_strides(q[0])
    d.grad_dtype = d.dtype
    return (ctypes.byref(d), *_sized(q[3], (oases_attn_workspace_bytes, d, False)),
            (d.batch, d.heads, d.q_len))


@functools.lru_cache(maxsize=512)
def _attn_bwd_plan(q, k, v, o, lse, do, outs, kv_lens, q_start, bias, dbias, need_dbias, *options):
    d = AttnDesc(**_attn_common(q, k, v, kv_lens, q_start, bias, *options))
    d.o, d.d_o = _heads_of("o", o, _like(q)), _heads_of("do", do, _like(q))
    _match("lse", lse, (d.batch, d.heads, d.q_len), torch.float32, q[3])
    for name, like, given in zip(("dq", "dk", "dv"), (q, k, v), outs):
        setattr(d, name, _row_strides(like[0]) if given is None
                else _heads_of(name, given, _like(like)))
    if dbias is not None:
        _need(bias is not None and need_dbias, "dbias is given, but there is none to form")
        _match("dbias", dbias, tuple(bias[0]), torch.float32, q[3])
    d.accumulate = int(dbias is not None)
    d.grad_dtype = 0 if dbias is not None else d.dtype
    return ctypes.byref(d), *_sized(q[3], (oases_attn_workspace_bytes, d, True))


def _out(x: Optional[torch.Tensor], given: Optional[torch.Tensor]):
    return torch.empty_like(x, memory_format=torch.contiguous_format) \
        if given is None and x is not None else given


def _whole(name: str, v) -> int:
    if isinstance(v, int):
        return int(v)
    try:
        n = int(v)
    except (TypeError, OverflowError, ValueError):
        n = None
    _need(n is not None and n == v, "%s must be a whole number, got %r" % (name, v))
    return n


def _start(q_start):
    """(the tensor or None, the number)"""
    if q_start is None:
        return None, 0
    return (q_start, 0) if isinstance(q_start, torch.Tensor) else (None, _whole("q_start", q_start))


def _options(causal, start, scale, max_distance, bidirectional):
    return (bool(causal), start, None if scale is None else float(scale),
            _whole("max_distance", max_distance),
            not causal if bidirectional is None else bool(bidirectional))


def attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
             kv_lens: Optional[torch.Tensor] = None, causal: bool = False,
             q_start: Union[int, torch.Tensor, None] = None, scale: Optional[float] = None,
             bias: Optional[torch.Tensor] = None, max_distance: int = 128,
             bidirectional: Optional[bool] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Softmax attention of q over keys of another length: (o, lse).

    q [batch, q_len, heads, head_dim], k and v [batch, k_len, kv_heads, head_dim],
    each with strides of its own; heads a multiple of kv_heads (query head h reads key
    head h // (heads // kv_heads)).  kv_lens int32 [batch]: how many keys each sequence
    has (default k_len); what stands behind them (causal: and behind the last query's
    position) is not used.  causal: key j is visible
    where j <= q_start + i; q_start: the first query's position, a number for all
    sequences or int32 [batch] (a single token behind a cache: its length - 1).  A cache that
    grows is best given whole, with kv_lens and q_start as tensors: a slice of another length
    or another number is another combination, checked anew (61 us of the host against 17).
    Up to four rows (q_len times heads // kv_heads) run on a kernel that reads each key once;
    beyond, a key is read by every query head that shares it.  scale: default head_dim ** -0.5.  bias [buckets, heads]: learned by the bucket of the
    key's position relative to the query's, as oases_attn.h defines it;
    bidirectional: default not causal.
    Returns o (contiguous, q's type) and lse, float32 [batch, heads, q_len]; a query
    without visible keys has o = 0 and lse = -inf.
    """
    _no_graph("attn_fwd", q, k, v, bias)
    start, number = _start(q_start)
    desc, n_ws, stat = _attn_fwd_plan(
        _view(q), _view(k), _view(v), _sig(kv_lens), _sig(start), _sig(bias),
        *_options(causal, number, scale, max_distance, bidirectional))
    o = torch.empty_like(q, memory_format=torch.contiguous_format)
    lse = q.new_empty(stat, dtype=torch.float32)
    _call(lib().oases_attn_fwd, q.get_device(), n_ws, desc, _ptr(q), _ptr(k), _ptr(v),
          _ptr(kv_lens), _ptr(start), _ptr(bias), _ptr(o), _ptr(lse))
    return o, lse


def attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
             lse: torch.Tensor, do: torch.Tensor, kv_lens: Optional[torch.Tensor] = None,
             causal: bool = False, q_start: Union[int, torch.Tensor, None] = None,
             scale: Optional[float] = None, bias: Optional[torch.Tensor] = None,
             max_distance: int = 128, bidirectional: Optional[bool] = None,
             out: Tuple[Optional[torch.Tensor], ...] = _NO_OUT,
             dbias: Optional[torch.Tensor] = None, need_dbias: bool = True
             ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Gradients (dq, dk, dv, dbias) of attn_fwd for the gradient do of o, with the same
    arguments and what it returned.

    out: tensors for dq, dk and dv, any of which may be None (allocated, contiguous);
    slices of one buffer give the packed projection's gradient.  dk and dv are 0
    behind kv_lens.  dbias None: returned in bias's type (None where there is no bias
    or need_dbias is false).  dbias a float32 [buckets, heads] tensor: it is added to
    (+=) and returned.
    """
    start, number = _start(q_start)
    desc, n_ws = _attn_bwd_plan(
        _view(q), _view(k), _view(v), _view(o), _sig(lse), _view(do), _NO_OUT if out is _NO_OUT else tuple(map(_view, out)),
        _sig(kv_lens), _sig(start), _sig(bias), _sig(dbias), bool(need_dbias),
        *_options(causal, number, scale, max_distance, bidirectional))
    dq, dk, dv = _out(q, out[0]), _out(k, out[1]), _out(v, out[2])
    if dbias is None and bias is not None and need_dbias:
        dbias = torch.empty_like(bias)
    _call(lib().oases_attn_bwd, q.get_device(), n_ws, desc, _ptr(q), _ptr(k), _ptr(v),
          _ptr(kv_lens), _ptr(start), _ptr(bias), _ptr(o), _ptr(lse), _ptr(do), _ptr(dq), _ptr(dk),
          _ptr(dv), _ptr(dbias))
    return dq, dk, dv, dbias


# ---- norms per head with the position rotation ------------------------------------------
def _qknorm_common(q, k, cos, sin, positions, wq, wk, eps, interleaved):
    sq = _heads_of("q", q)
    (B, S, H, D), dtype, dev = _like(q)
    G = 0
    sk = Strides(0, 0, 0)
    if k is not None:
        _need(len(k[0]) == 4, "k must be a [batch, tokens, heads, head_dim] tensor")
        G = k[0][2]
        sk = _heads_of("k", k, ((B, S, G, D), dtype, dev))
    for name, w in (("q_weight", wq), ("k_weight", wk)):
        if w is not None:
            _match(name, w, (D,), dtype, dev)
    _need(k is not None or wk is None, "k_weight is given, but no k")
    _need((cos is None) == (sin is None), "cos and sin belong together")
    P = rot = shared = 0
    if cos is not None:
        _need(len(cos[0]) == 2, "cos must be [positions, rot / 2]")
        P, rot = cos[0][0], 2 * cos[0][1]
        _fits(positions=P, rot=rot)
        _need(rot <= D, "the tables turn %d values of %d" % (rot, D))
        for name, t in (("cos", cos), ("sin", sin)):
            _match(name, t, (P, rot // 2), torch.float32, dev)
        if positions is not None:
            shared = int(tuple(positions[0]) == (S,))
            _match("positions", positions, (S,) if shared else (B, S), torch.int64, dev)
        else:
            _need(rot == 0 or S <= P, "%d tokens, but the tables hold %d positions" % (S, P))
    else:
        _need(positions is None, "positions are given, but no tables")
    return dict(dtype=_CODE[dtype], batch=B, seq=S, heads=H, kv_heads=G, head_dim=D, rot=rot,
                interleaved=int(interleaved), positions_len=P, positions_shared=shared, eps=eps,
                q=sq, k=sk)


@functools.lru_cache(maxsize=512)
def _qknorm_fwd_plan(q, k, outs, *rest):
    d = QknormDesc(**_qknorm_common(q, k, *rest))
    d.grad_dtype = d.dtype
    for name, x, given in zip(("q_out", "k_out"), (q, k), outs):
        _need(x is not None or given is None, "out has a place for k, but there is no k")
        if x is not None:
            setattr(d, name, _row_strides(x[0]) if given is None
                    else _heads_of(name, given, _like(x)))
    return (ctypes.byref(d),)


@functools.lru_cache(maxsize=512)
def _qknorm_bwd_plan(q, k, dqo, dko, outs, grads, *rest):
    d = QknormDesc(**_qknorm_common(q, k, *rest))
    wq, wk = rest[3:5]
    d.q_out = _heads_of("dq_out", dqo, _like(q))
    _need((k is None) == (dko is None), "k and dk_out belong together")
    if k is not None:
        d.k_out = _heads_of("dk_out", dko, _like(k))
    for name, x, given in zip(("dq", "dk"), (q, k), outs):
        _need(x is not None or given is None, "out has a place for dk, but there is no k")
        if x is not None:
            setattr(d, name, _row_strides(x[0]) if given is None
                    else _heads_of(name, given, _like(x)))
    accumulate = grads is not None
    if accumulate:
        for name, g, w in zip(("dq_weight", "dk_weight"), grads, (wq, wk)):
            if g is not None:
                _need(w is not None, "%s has no weight" % name)
                _match(name, g, (d.head_dim,), torch.float32, q[3])
    d.accumulate = int(accumulate)
    d.grad_dtype = 0 if accumulate else d.dtype
    return ctypes.byref(d), *_sized(q[3], (oases_qknorm_workspace_bytes, d))


def qk_norm_rope_fwd(q: torch.Tensor, k: Optional[torch.Tensor], cos: Optional[torch.Tensor],
                     sin: Optional[torch.Tensor], positions: Optional[torch.Tensor] = None,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     interleaved: bool = False,
                     out: Tuple[Optional[torch.Tensor], ...] = (None, None)
                     ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Queries and keys, each head's values divided by their root mean square and times
    a weight, then turned by the angles of the token's position: (q', k').

    q [batch, seq, heads, head_dim] and k [batch, seq, kv_heads, head_dim] (or None),
    with strides of their own.  q_weight, k_weight [head_dim] (None: 1).  cos, sin
    float32 [positions, rot / 2] (None: no rotation) turn the first rot values of a
    head, in pairs (c, c + rot / 2) or, interleaved, (2c, 2c + 1).  positions int64
    [batch, seq] or [seq]: rows of the tables (None: token t is at t); one outside them
    makes its token's rotated values NaN.
    out: tensors for q' and k' (None: allocated, contiguous); q and k themselves for
    the rotation in place.
    """
    _no_graph("qk_norm_rope_fwd", q, k, q_weight, k_weight)
    (desc,) = _qknorm_fwd_plan(
        _view(q), _view(k), tuple(map(_view, out)), _sig(cos), _sig(sin), _sig(positions),
        _sig(q_weight), _sig(k_weight), float(eps), bool(interleaved))
    qo, ko = _out(q, out[0]), _out(k, out[1])
    _call_no_ws(lib().oases_qknorm_fwd, q.get_device(), desc, _ptr(q), _ptr(k), _ptr(cos),
                _ptr(sin), _ptr(positions), _ptr(q_weight), _ptr(k_weight), _ptr(qo), _ptr(ko))
    return qo, ko


def qk_norm_rope_bwd(q: torch.Tensor, k: Optional[torch.Tensor], dq_out: torch.Tensor,
                     dk_out: Optional[torch.Tensor], cos: Optional[torch.Tensor],
                     sin: Optional[torch.Tensor], positions: Optional[torch.Tensor] = None,
                     q_weight: Optional[torch.Tensor] = None,
                     k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                     interleaved: bool = False,
                     out: Tuple[Optional[torch.Tensor], ...] = (None, None),
                     grads: Optional[Tuple[Optional[torch.Tensor], ...]] = None):
    """Gradients (dq, dk, dq_weight, dk_weight) of qk_norm_rope_fwd, whose q and k these
    are, for the gradients dq_out and dk_out of its outputs.

    out: tensors for dq and dk (None: allocated; dq_out and dk_out themselves for the
    gradient in place).  grads None: the gradients of the weights given are returned in
    their type (None where there is no weight).  grads a pair of float32 [head_dim]
    tensors, either None (left out): they are added to (+=), and returned.
    """
    desc, n_ws = _qknorm_bwd_plan(
        _view(q), _view(k), _view(dq_out), _view(dk_out), tuple(map(_view, out)),
        None if grads is None else tuple(map(_sig, grads)), _sig(cos), _sig(sin), _sig(positions),
        _sig(q_weight), _sig(k_weight), float(eps), bool(interleaved))
    dq, dk = _out(q, out[0]), _out(k, out[1])
    dwq, dwk = grads if grads is not None else (
        None if w is None else torch.empty_like(w) for w in (q_weight, k_weight))
    _call(lib().oases_qknorm_bwd, q.get_device(), n_ws, desc, _ptr(q), _ptr(k), _ptr(dq_out),
          _ptr(dk_out), _ptr(cos), _ptr(sin), _ptr(positions), _ptr(q_weight), _ptr(k_weight),
          _ptr(dq), _ptr(dk), _ptr(dwq), _ptr(dwk))
    return dq, dk, dwq, dwk


__all__ = ["glu_fwd", "glu_bwd", "ce_fwd", "ce_bwd", "attn_fwd", "attn_bwd", "qk_norm_rope_fwd",
           "qk_norm_rope_bwd"]
