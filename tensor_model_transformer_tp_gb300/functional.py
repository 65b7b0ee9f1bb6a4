"""The gated feed-forward block and the linear head's cross entropy on torch tensors.

Each function checks its tensors (once per combination of shapes, types and
options), allocates outputs and workspace with torch's caching allocator and makes
one call of liboases.so on torch's current stream of the tensors' device; nothing
is computed here and no data is kept between calls.  Because the allocations
follow torch's stream rules, the calls can be made on any stream, from several
threads, and inside CUDA graph capture.

Tensors are contiguous, on one CUDA device, ``float32`` or ``bfloat16`` as
``x`` is; anything else raises ``ValueError`` before a call is made.  Errors of
the library raise ``OasesError``.  There is no autograd integration: the
backward functions are called with what the forward returned.  (A forward function
given a tensor that requires a gradient, in grad mode, warns of it once.)
"""
from __future__ import annotations

import ctypes
import functools
import warnings
from typing import Dict, Optional, Tuple

import torch

from . import (ACT, KEEP, CeDesc, GluDesc, GluGrads, GluWeights, _check as _check_status, lib,
               oases_ce_workspace_bytes, oases_glu_saved_bytes, oases_glu_workspace_bytes)

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


__all__ = ["glu_fwd", "glu_bwd", "ce_fwd", "ce_bwd"]
