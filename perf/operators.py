"""Workloads of the training-head and gated feed-forward operators.

Two families of operators are measured, each in its forward form and as a
training pass (forward and backward):

glu   the gated feed-forward block  y = (act(x Wg^T + bg) * (x Wu^T + bu)) W2^T + b2 (+ resid),
      with w1 = [Wg; Wu] stacked as [2 * ffn, hidden].  Its training pass keeps
      between forward and backward either nothing ("none": the backward
      recomputes both projections), the two projections in the storage type
      ("pre"), or the two projections in 8 bits ("mxfp8": E4M3 codes and one
      power-of-two scale per 32 consecutive columns of each projection, scale
      exponent floor(log2 max|v|) - 8; the backward then uses those values).
ce    softmax cross entropy of the linear head logits = x W^T over a large
      vocabulary, per token loss[m] = logsumexp(logits[m]) - logits[m, target];
      rows whose target is IGNORE have loss 0 and no gradient.  Its training
      pass takes the gradient of the loss (one value for all rows, or one per
      row) and returns the gradients of x and W.

``own`` False: elementary torch operations in 32 bits, rounded once at the end.
``own`` True: the calls a user makes of tensor_model_transformer_tp_gb300.functional.
"""
import math

import torch

own = False

IGNORE = -100
BLOCK = 32          # columns per scale of the 8-bit form
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def _glu(name, op, dtype, rows, hidden, ffn, act, save="none", bias=False, resid=False):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "hidden": hidden, "ffn": ffn,
            "act": act, "save": save, "bias": bias, "resid": resid}


def _ce(name, op, dtype, rows, hidden, vocab, per_row=False):
    return {"name": name, "op": op, "dtype": dtype, "rows": rows, "hidden": hidden, "vocab": vocab,
            "per_row": per_row}


def listed():
    return [
        # one token of a model being sampled: bound by reading the weights once
        _glu("glu fwd, one token", "glu_fwd", "bf16", 1, 2560, 6912, "silu", resid=True),
        # a few sequences' next tokens, or a short prompt: small, ragged, with biases
        _glu("glu fwd, 61 rows", "glu_fwd", "bf16", 61, 1024, 2736, "silu", bias=True, resid=True),
        # evaluation of a layer over full sequences
        _glu("glu fwd, 4096 rows", "glu_fwd", "bf16", 4096, 4096, 11008, "silu", resid=True),
        # a small model in 32 bits, where the launches count
        _glu("glu train, f32", "glu_train", "f32", 256, 256, 1024, "gelu", save="pre", bias=True),
        # the feed-forward workload of this repository's hidden size 1024
        _glu("glu train, kept", "glu_train", "bf16", 4096, 1024, 4096, "silu", save="pre"),
        # packed sequences of odd total length, both projections recomputed
        _glu("glu train, recomputed", "glu_train", "bf16", 1531, 2048, 5464, "gelu", save="none",
             bias=True, resid=True),
        # one sub-batch of the four-layer stack, projections kept in 8 bits
        _glu("glu train, kept in 8 bits", "glu_train", "bf16", 8192, 2560, 10240, "silu",
             save="mxfp8"),
        # scoring the last tokens of a few sequences
        _ce("ce fwd, 37 rows", "ce_fwd", "bf16", 37, 1024, 50257),
        # validation loss over full sequences
        _ce("ce fwd, 4096 rows", "ce_fwd", "bf16", 4096, 4096, 32000),
        # a small model in 32 bits with a character-level vocabulary
        _ce("ce train, f32", "ce_train", "f32", 250, 256, 1003),
        # packed sequences of odd total length, per-token loss weights
        _ce("ce train, 2041 rows", "ce_train", "bf16", 2041, 1024, 50257, per_row=True),
        # the head behind one sub-batch of the four-layer stack, mean loss
        _ce("ce train, 8192 rows", "ce_train", "bf16", 8192, 2560, 50304),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    op = rng.choice(["glu_fwd", "glu_train", "ce_fwd", "ce_train"])
    small = rng.random() < 0.2            # the 32-bit types serve small models
    dtype = "f32" if small else "bf16"
    hidden = _log_int(rng, 64, 1024, 1) if small else _log_int(rng, 256, 4096, 8)
    if op.startswith("glu"):
        ffn = _log_int(rng, 96, 2048, 1) if small else _log_int(rng, 512, 12288, 8)
        most = 512 if small else max(1, min(8192, 8192 * 2560 * 10240 // (hidden * ffn)))
        return {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, most), "hidden": hidden,
                "ffn": ffn, "act": rng.choice(["silu", "gelu"]),
                # the 8-bit form is kept beside bf16 storage only
                "save": "none" if op == "glu_fwd" else
                        rng.choice(["none", "pre"] if small else ["none", "pre", "mxfp8"]),
                "bias": rng.random() < 0.5, "resid": rng.random() < 0.5}
    vocab = _log_int(rng, 200, 8000) if small else _log_int(rng, 1000, 131072)
    most = 512 if small else max(1, min(8192, 8192 * 50304 * 2560 // (hidden * vocab),
                                        8192 * 50304 // vocab))
    return {"op": op, "dtype": dtype, "rows": _log_int(rng, 1, most), "hidden": hidden,
            "vocab": vocab, "per_row": rng.random() < 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t = DTYPES[case["dtype"]]
    M, H = case["rows"], case["hidden"]

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * std).to(t)

    state = {"case": case, "x": normal(M, H)}       # x: the rows after a normalisation
    if case["op"].startswith("glu"):
        F = case["ffn"]
        state["weights"] = {"w1": normal(2 * F, H, std=0.02), "w2": normal(H, F, std=0.02)}
        if case["bias"]:
            state["weights"] |= {"b1": normal(2 * F, std=0.02), "b2": normal(H, std=0.02)}
        state["resid"] = normal(M, H) if case["resid"] else None
        if case["op"] == "glu_train":
            state["dy"] = normal(M, H)
        return state
    V = case["vocab"]
    state["w"] = normal(V, H, std=0.02)
    # token frequencies fall off steeply, so the same targets recur; a tenth of
    # the rows (padding, prompts) carry no loss
    u = torch.rand(M, generator=gen, device="cuda", dtype=torch.float64)
    state["targets"] = (u ** 3 * V).long().clamp_(max=V - 1)
    ignored = torch.rand(M, generator=gen, device="cuda") < 0.1
    state["targets"][ignored] = IGNORE
    n = max(1, M)
    if case["per_row"]:
        state["dloss"] = (0.5 + torch.rand(M, generator=gen, device="cuda")) / n
    else:
        state["dloss"] = torch.full((1,), 1.0 / n, device="cuda")
    return state


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    M, H = case["rows"], case["hidden"]
    train = case["op"].endswith("train")
    if case["op"].startswith("glu"):
        F = case["ffn"]
        params = 3 * H * F + ((2 * F + H) if case["bias"] else 0)
        rows = M * H * (2 + (1 if case["resid"] else 0) + (2 if train else 0))
        return {"bytes": e * (rows + params * (2 if train else 1)),
                "flops": 6.0 * M * H * F * (3 if train else 1)}
    V = case["vocab"]
    n = e * (M * H + V * H) * (2 if train else 1) + 8 * M + 8 * M   # targets, loss and lse
    n += 4 * M if train and case["per_row"] else 0
    return {"bytes": n, "flops": 2.0 * M * V * H * (3 if train else 1)}


# ---- the framework's operators ------------------------------------------------
def _run_own(s):
    from tensor_model_transformer_tp_gb300 import functional as F

    c = s["case"]
    if c["op"].startswith("glu"):
        y, saved = F.glu_fwd(s["x"], s["weights"], act=c["act"], resid=s["resid"], save=c["save"])
        if c["op"] == "glu_fwd":
            return {"y": y}
        dx, grads = F.glu_bwd(s["x"], s["dy"], s["weights"], act=c["act"], save=c["save"],
                              saved=saved)
        return {"y": y, "dx": dx, "grads": grads}
    loss, lse = F.ce_fwd(s["x"], s["w"], s["targets"], ignore_index=IGNORE)
    if c["op"] == "ce_fwd":
        return {"loss": loss, "lse": lse}
    dx, dw = F.ce_bwd(s["x"], s["w"], s["targets"], lse, s["dloss"], ignore_index=IGNORE)
    return {"loss": loss, "lse": lse, "dx": dx, "dw": dw}


# ---- the plain form -------------------------------------------------------------
def _act(a, kind):
    """act(a) and its derivative."""
    if kind == "silu":
        p = 1.0 / (1.0 + torch.exp(-a))
        return a * p, p * (1.0 + a * (1.0 - p))
    cdf = 0.5 * (1.0 + torch.erf(a * math.sqrt(0.5)))
    return a * cdf, cdf + a * torch.exp(-0.5 * a * a) / math.sqrt(2.0 * math.pi)


def _eight_bits(v):
    """The values that v [M, F] has in E4M3 with one scale per 32 columns."""
    M, F = v.shape
    n = (F + BLOCK - 1) // BLOCK
    b = torch.zeros(M, n * BLOCK, device=v.device)
    b[:, :F] = v
    b = b.view(M, n, BLOCK)
    amax = b.abs().amax(dim=2, keepdim=True)
    _, e = torch.frexp(amax)                       # amax = f * 2^e, f in [0.5, 1)
    e = torch.where(amax > 0, (e - 1 - 8).clamp(-127, 127), torch.zeros_like(e))
    q = torch.ldexp(b, -e).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).float()
    return torch.ldexp(q, e).view(M, n * BLOCK)[:, :F]


def _run_plain(s):
    c = s["case"]
    t = DTYPES[c["dtype"]]
    x = s["x"].float()
    if c["op"].startswith("glu"):
        F, w = c["ffn"], {k: v.float() for k, v in s["weights"].items()}
        p = x @ w["w1"].t()
        if c["bias"]:
            p = p + w["b1"]
        a, b = p[:, :F], p[:, F:]
        y = (_act(a, c["act"])[0] * b) @ w["w2"].t()
        if c["bias"]:
            y = y + w["b2"]
        if c["resid"]:
            y = y + s["resid"].float()
        if c["op"] == "glu_fwd":
            return {"y": y.to(t)}
        if c["save"] == "mxfp8":
            a, b = _eight_bits(a), _eight_bits(b)
        dy = s["dy"].float()
        f, df = _act(a, c["act"])
        dh = dy @ w["w2"]
        dp = torch.cat([dh * b * df, dh * f], dim=1)
        grads = {"w1": (dp.t() @ x).to(t), "w2": (dy.t() @ (f * b)).to(t)}
        if c["bias"]:
            grads |= {"b1": dp.sum(dim=0).to(t), "b2": dy.sum(dim=0).to(t)}
        return {"y": y.to(t), "dx": (dp @ w["w1"]).to(t), "grads": grads}
    w, target = s["w"].float(), s["targets"]
    logits = x @ w.t()
    top = logits.amax(dim=1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(dim=1))
    used = target != IGNORE
    at = torch.where(used, target, torch.zeros_like(target))
    rows = torch.arange(x.shape[0], device=x.device)
    loss = torch.where(used, lse - logits[rows, at], torch.zeros_like(lse))
    if c["op"] == "ce_fwd":
        return {"loss": loss, "lse": lse}
    g = torch.exp(logits - lse[:, None])
    g[rows, at] -= 1.0
    g = g * torch.where(used, s["dloss"].expand_as(lse), torch.zeros_like(lse))[:, None]
    return {"loss": loss, "lse": lse, "dx": (g @ w).to(t), "dw": (g.t() @ x).to(t)}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits ----------------------------------------------------
def _e4m3_blocks_64(v):
    """v rounded to the 8-bit form, from the format's definition: magnitudes
    (8 + m) 2^(q - 3) with m < 8 and q >= -6, steps of 2^-9 below 2^-6, largest
    448, nearest value with ties to the even one."""
    out = torch.empty_like(v)
    for j in range(0, v.shape[1], BLOCK):
        b = v[:, j:j + BLOCK]
        top = b.abs().max(dim=1, keepdim=True).values
        scale = torch.where(top > 0, torch.exp2(torch.floor(torch.log2(top)) - 8.0),
                            torch.ones_like(top))
        r = b / scale
        q = torch.floor(torch.log2(r.abs().clamp_min(2.0 ** -6)))
        step = torch.exp2(q - 3.0)
        out[:, j:j + BLOCK] = (torch.round(r / step) * step).clamp(-448.0, 448.0) * scale
    return out


def exact(case, seed):
    s = prepare(case, seed)
    wide = lambda v: v.double().requires_grad_(True)  # noqa: E731
    x = wide(s["x"])
    if case["op"].startswith("glu"):
        F = case["ffn"]
        act = torch.nn.functional.silu if case["act"] == "silu" else torch.nn.functional.gelu
        w = {k: wide(v) for k, v in s["weights"].items()}
        p = torch.nn.functional.linear(x, w["w1"], w.get("b1"))
        y = torch.nn.functional.linear(act(p[:, :F]) * p[:, F:], w["w2"], w.get("b2"))
        if s["resid"] is not None:
            y = y + s["resid"].double()
        if case["op"] == "glu_fwd":
            return {"y": y.detach()}
        dy = s["dy"].double()
        names = list(w)
        if case["save"] != "mxfp8":
            got = torch.autograd.grad(y, [x] + [w[k] for k in names], dy)
        else:
            # the backward pass at the values that were kept
            k8 = torch.cat([_e4m3_blocks_64(p.detach()[:, :F]), _e4m3_blocks_64(p.detach()[:, F:])],
                           dim=1).requires_grad_(True)
            y8 = torch.nn.functional.linear(act(k8[:, :F]) * k8[:, F:], w["w2"], w.get("b2"))
            late = [k for k in names if k in ("w2", "b2")]
            part = torch.autograd.grad(y8, [k8] + [w[k] for k in late], dy)
            early = [k for k in names if k in ("w1", "b1")]
            rest = torch.autograd.grad(p, [x] + [w[k] for k in early], part[0])
            by = dict(zip(late, part[1:])) | dict(zip(early, rest[1:]))
            got = [rest[0]] + [by[k] for k in names]
        return {"y": y.detach(), "dx": got[0], "grads": dict(zip(names, got[1:]))}
    w = wide(s["w"])
    logits = torch.nn.functional.linear(x, w)
    loss = torch.nn.functional.cross_entropy(logits, s["targets"], ignore_index=IGNORE,
                                             reduction="none")
    lse = torch.logsumexp(logits.detach(), dim=1)
    if case["op"] == "ce_fwd":
        return {"loss": loss.detach(), "lse": lse}
    dx, dw = torch.autograd.grad(loss, [x, w], s["dloss"].double().expand_as(loss))
    return {"loss": loss.detach(), "lse": lse, "dx": dx, "dw": dw}
