"""The gated feed-forward block and the linear head's cross entropy on torch tensors.

Each function checks its tensors, allocates outputs and workspace with torch's
allocator and makes one call of liboases.so on torch's current stream of the
tensors' device; nothing is computed here and nothing is kept between calls.
Because the allocations follow torch's stream rules, the calls can be made on
any stream, from several threads, and inside CUDA graph capture.

Tensors are contiguous, on one CUDA device, ``float32`` or ``bfloat16`` as
``x`` is; anything else raises ``ValueError`` before a call is made.  Errors of
the library raise ``OasesError``.  There is no autograd integration: the
backward functions are called with what the forward returned.
"""
from __future__ import annotations

import functools
from typing import Dict, Optional, Tuple

import torch

from . import (ACT, KEEP, CeDesc, GluDesc, GluGrads, GluWeights, oases_ce_bwd, oases_ce_fwd,
               oases_ce_workspace_bytes, oases_glu_bwd, oases_glu_fwd, oases_glu_saved_bytes,
               oases_glu_workspace_bytes)

_CODE = {torch.float32: 0, torch.bfloat16: 1}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _check(name: str, t: torch.Tensor, shape: tuple, dtype: torch.dtype, device) -> None:
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != shape:
        raise ValueError("%s must be a %s tensor of shape %s, got %s" % (
            name, dtype, shape, (t.dtype, tuple(t.shape)) if isinstance(t, torch.Tensor) else type(t)))
    if t.device != device:
        raise ValueError("%s is on %s, x on %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s is not contiguous" % name)


def _rows(x: torch.Tensor) -> Tuple[int, int]:
    _need(isinstance(x, torch.Tensor) and x.dim() == 2, "x must be a [rows, hidden] tensor")
    _need(x.dtype in _CODE, "x must be float32 or bfloat16, got %s" % x.dtype)
    _need(x.is_cuda, "x must be on a CUDA device, got %s" % x.device)
    _need(x.is_contiguous(), "x is not contiguous")
    return x.shape[0], x.shape[1]


class _on:
    """The tensors' device, current for the call."""

    def __init__(self, device):
        self.device = device

    def __enter__(self):
        self.guard = None
        if torch.cuda.current_device() != self.device.index:
            self.guard = torch.cuda.device(self.device)
            self.guard.__enter__()
        return torch.cuda.current_stream(self.device).cuda_stream

    def __exit__(self, *exc):
        if self.guard is not None:
            self.guard.__exit__(*exc)


def _bytes(n: int, device) -> Optional[torch.Tensor]:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


# ---- gated feed-forward block ---------------------------------------------------
@functools.lru_cache(maxsize=256)
def _glu_desc(dtype, rows, hidden, ffn, act, keep, dx_dtype, grad_dtype, accumulate):
    d = GluDesc(dtype, rows, hidden, ffn, act, keep, dx_dtype, grad_dtype, accumulate)
    return (d, oases_glu_saved_bytes(d), oases_glu_workspace_bytes(d, False),
            oases_glu_workspace_bytes(d, True))


def _glu_weights(x, weights: Dict[str, torch.Tensor], hidden: int):
    unknown = set(weights) - {"w1", "b1", "w2", "b2"}
    _need(not unknown, "unknown weights %s" % sorted(unknown))
    _need("w1" in weights and "w2" in weights, "weights needs w1 and w2")
    w2 = weights["w2"]
    _need(isinstance(w2, torch.Tensor) and w2.dim() == 2, "w2 must be [hidden, ffn]")
    ffn = w2.shape[1]
    shapes = {"w1": (2 * ffn, hidden), "b1": (2 * ffn,), "w2": (hidden, ffn), "b2": (hidden,)}
    for k, v in weights.items():
        if v is not None:
            _check(k, v, shapes[k], x.dtype, x.device)
    _need(weights["w1"] is not None, "weights needs w1 and w2")
    return ffn, shapes


def glu_fwd(x: torch.Tensor, weights: Dict[str, torch.Tensor], act: str = "silu",
            resid: Optional[torch.Tensor] = None, save: str = "none",
            y: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """y = (act(x Wg^T + bg) * (x Wu^T + bu)) W2^T + b2 (+ resid).

    x [rows, hidden]; weights: "w1" [2 ffn, hidden] = [Wg; Wu], "w2"
    [hidden, ffn] and optionally "b1" [2 ffn], "b2" [hidden].  act: "silu" or
    "gelu" (exact).  save: what is kept for the backward beside x: "none",
    "pre" ([a | b], [rows, 2 ffn] in x's type) or "mxfp8" (a and b in 8 bits, a
    byte tensor in the layout of oases_glu.h; bfloat16 only).
    Returns (y, kept activations or None).  y may be given (resid itself, for
    an in-place residual).
    """
    rows, hidden = _rows(x)
    ffn, _ = _glu_weights(x, weights, hidden)
    _need(act in ACT, "act must be one of %s" % sorted(ACT))
    _need(save in KEEP, "save must be one of %s" % sorted(KEEP))
    if resid is not None:
        _check("resid", resid, (rows, hidden), x.dtype, x.device)
    if y is None:
        y = torch.empty_like(x)
    else:
        _check("y", y, (rows, hidden), x.dtype, x.device)
    t = _CODE[x.dtype]
    desc, n_saved, n_ws, _ = _glu_desc(t, rows, hidden, ffn, ACT[act], KEEP[save], t, t, 0)
    saved = None
    if save == "pre":
        saved = torch.empty((rows, 2 * ffn), dtype=x.dtype, device=x.device)
    elif save == "mxfp8":
        saved = torch.empty(n_saved, dtype=torch.uint8, device=x.device)
    with _on(x.device) as stream:
        oases_glu_fwd(desc, GluWeights.of(weights), x, resid, y, saved, _bytes(n_ws, x.device),
                      n_ws, stream)
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
    rows, hidden = _rows(x)
    ffn, shapes = _glu_weights(x, weights, hidden)
    _need(act in ACT, "act must be one of %s" % sorted(ACT))
    _need(save in KEEP, "save must be one of %s" % sorted(KEEP))
    _check("dy", dy, (rows, hidden), x.dtype, x.device)
    accumulate = grads is not None
    if accumulate:
        for k, v in grads.items():
            _need(weights.get(k) is not None, "grads[%r] has no weight" % k)
            _check("grads[%r]" % k, v, shapes[k], torch.float32, x.device)
    else:
        grads = {k: torch.empty_like(v) for k, v in weights.items() if v is not None}
    dx_dtype = x.dtype if dx_dtype is None else dx_dtype
    _need(dx_dtype in (x.dtype, torch.float32), "dx_dtype must be x's type or float32")
    t = _CODE[x.dtype]
    desc, n_saved, _, n_ws = _glu_desc(t, rows, hidden, ffn, ACT[act], KEEP[save], _CODE[dx_dtype],
                                       0 if accumulate else t, int(accumulate))
    if save == "none":
        _need(saved is None, "saved is given, but save is \"none\"")
    elif save == "pre":
        _check("saved", saved, (rows, 2 * ffn), x.dtype, x.device)
    else:
        _check("saved", saved, (n_saved,), torch.uint8, x.device)
    dx = torch.empty((rows, hidden), dtype=dx_dtype, device=x.device) if need_dx else None
    with _on(x.device) as stream:
        oases_glu_bwd(desc, GluWeights.of(weights), x, dy, saved, dx, GluGrads.of(grads),
                      _bytes(n_ws, x.device), n_ws, stream)
    return dx, grads


# ---- cross entropy of the linear head -----------------------------------------------
@functools.lru_cache(maxsize=256)
def _ce_desc(ignore_index, dtype, rows, hidden, vocab, per_row, grad_dtype, accumulate):
    d = CeDesc(ignore_index, dtype, rows, hidden, vocab, per_row, grad_dtype, accumulate)
    return d, oases_ce_workspace_bytes(d, False), oases_ce_workspace_bytes(d, True)


def _ce_check(x, w, targets):
    rows, hidden = _rows(x)
    _need(isinstance(w, torch.Tensor) and w.dim() == 2 and w.shape[0] > 0,
          "w must be a [vocab, hidden] tensor")
    _check("w", w, (w.shape[0], hidden), x.dtype, x.device)
    _check("targets", targets, (rows,), torch.int64, x.device)
    return rows, hidden, w.shape[0]


def ce_fwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor,
           ignore_index: int = -100) -> Tuple[torch.Tensor, torch.Tensor]:
    """Per-row cross entropy of the logits x w^T: (loss, lse), float32 [rows].

    x [rows, hidden], w [vocab, hidden], targets int64 [rows].  Rows whose
    target is ignore_index have loss 0; another target outside [0, vocab)
    gives NaN.  The logits are not kept.
    """
    rows, hidden, vocab = _ce_check(x, w, targets)
    t = _CODE[x.dtype]
    desc, n_ws, _ = _ce_desc(ignore_index, t, rows, hidden, vocab, 0, t, 0)
    loss = torch.empty(rows, dtype=torch.float32, device=x.device)
    lse = torch.empty(rows, dtype=torch.float32, device=x.device)
    with _on(x.device) as stream:
        oases_ce_fwd(desc, x, w, targets, loss, lse, _bytes(n_ws, x.device), n_ws, stream)
    return loss, lse


def ce_bwd(x: torch.Tensor, w: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
           dloss: torch.Tensor, dw: Optional[torch.Tensor] = None, ignore_index: int = -100,
           need_dx: bool = True, need_dw: bool = True
           ) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """Gradients (dx, dw) of ce_fwd for the gradient dloss of its losses:
    float32, [rows], or [1] (or a scalar tensor) for the same value in every row
    (1 / n for the mean over n rows with a loss).

    dw None: returned in x's type.  dw a float32 [vocab, hidden] tensor: it is
    added to (+=) and returned.
    """
    rows, hidden, vocab = _ce_check(x, w, targets)
    _check("lse", lse, (rows,), torch.float32, x.device)
    _need(isinstance(dloss, torch.Tensor), "dloss must be a tensor")
    per_row = tuple(dloss.shape) not in ((), (1,))
    _check("dloss", dloss, (rows,) if per_row else tuple(dloss.shape), torch.float32, x.device)
    accumulate = dw is not None
    _need(need_dw or not accumulate, "dw is given, but need_dw is false")
    if accumulate:
        _check("dw", dw, (vocab, hidden), torch.float32, x.device)
    elif need_dw:
        dw = torch.empty_like(w)
    t = _CODE[x.dtype]
    desc, _, n_ws = _ce_desc(ignore_index, t, rows, hidden, vocab, int(per_row),
                             0 if accumulate else t, int(accumulate))
    dx = torch.empty_like(x) if need_dx else None
    with _on(x.device) as stream:
        oases_ce_bwd(desc, x, w, targets, lse, dloss, dx, dw, _bytes(n_ws, x.device), n_ws, stream)
    return dx, dw


__all__ = ["glu_fwd", "glu_bwd", "ce_fwd", "ce_bwd"]
