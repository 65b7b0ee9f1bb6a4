"""Workloads of the attention operators beside the block's own causal attention.

Two families, each in its forward form and as a training pass (forward and
backward):

attn  softmax attention of q [B, Sq, H, D] over k, v [B, Sk, Hkv, D] of another
      length: s = scale q k^T + bias, key j of sequence b counts where
      j < kv_lens[b] and, where causal, j <= q_start[b] + i; a query without keys
      gets 0 (and lse -inf) and gives no gradient.  H is a multiple of Hkv: query
      head h reads key head h // (H / Hkv).  The bias is learned by relative
      position: table[bucket(n), h] with n = j - (q_start[b] + i), and its
      gradient is the sum of ds over each bucket.
        bucket(n): N buckets for each sign (bidirectional: N = buckets / 2, keys
        after the query in the upper half) or for the past alone (N = buckets,
        keys after the query as at distance 0); with a = |n|, E = N // 2:
        a where a < E, else min(N - 1, E + floor((N - E) log(a / E) / log(max_distance / E))).
qk    per head, over the D values of each query and key: x / sqrt(mean x^2 + eps)
      times a weight [D], then a rotation of the first R values by the position's
      angles: cos and sin tables [positions, R / 2], pairs (c, c + R / 2) or, where
      interleaved, (2c, 2c + 1).  The training pass returns the gradients of the
      unnormalised queries and keys and of both weights.

``own`` False: elementary torch operations in 32 bits, rounded once at the end.
``own`` True: the calls a user makes of tensor_model_transformer_tp_gb300.functional.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
EPS = 1e-6


def _qk(name, dtype, batch, seq, heads, kv_heads, dim, rot, train, interleaved=False):
    return {"name": name, "op": "qk", "dtype": dtype, "batch": batch, "seq": seq, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "train": train, "interleaved": interleaved}


def _attn(name, dtype, batch, q_len, k_len, heads, kv_heads, dim, train, ragged=False, causal=False,
          buckets=0, max_distance=128):
    return {"name": name, "op": "attn", "dtype": dtype, "batch": batch, "q_len": q_len,
            "k_len": k_len, "heads": heads, "kv_heads": kv_heads, "dim": dim, "train": train,
            "ragged": ragged, "causal": causal, "buckets": buckets, "max_distance": max_distance}


def listed():
    return [
        # the next tokens of 64 sequences being sampled, at their own far positions
        _qk("qk norm fwd, next tokens", "bf16", 64, 1, 32, 8, 128, 128, False),
        # one sub-batch of the four-layer stack (hidden 2560, 20 heads)
        _qk("qk norm train, 8192 tokens", "bf16", 4, 2048, 20, 20, 128, 128, True),
        # a small model in 32 bits: grouped heads, part of each head rotated
        _qk("qk norm train, f32", "f32", 3, 171, 6, 2, 80, 32, True, interleaved=True),
        # a decoder's next token over the encoder's states of 16 sequences
        _attn("cross fwd, one token", "bf16", 16, 1, 1500, 20, 20, 64, False, ragged=True),
        # a few latent queries over one long sequence of states
        _attn("cross fwd, 64 queries, long", "bf16", 1, 64, 32768, 16, 16, 128, False),
        # an encoder-decoder's training step, padded sources, odd lengths
        _attn("cross train, padded", "bf16", 8, 509, 1531, 16, 16, 64, True, ragged=True),
        # long sources, key heads shared by four query heads
        _attn("cross train, grouped heads", "bf16", 2, 2048, 4096, 32, 8, 128, True),
        # a small model in 32 bits
        _attn("cross train, f32", "f32", 4, 50, 77, 8, 8, 32, True, ragged=True),
        # the next token of a decoder whose layers carry a relative position bias
        _attn("bias fwd, one token", "bf16", 32, 1, 1024, 12, 12, 64, False, ragged=True,
              causal=True, buckets=32),
        # an encoder of the four-layer stack's sizes: both directions
        _attn("bias train, both directions", "bf16", 4, 2048, 2048, 20, 20, 128, True, buckets=32),
        # a decoder's training step on ragged sequences
        _attn("bias train, causal", "bf16", 3, 777, 777, 12, 12, 64, True, ragged=True, causal=True,
              buckets=32),
        # a small model in 32 bits
        _attn("bias train, f32", "f32", 2, 130, 130, 6, 6, 64, True, buckets=32),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step))


def draw(rng):
    small = rng.random() < 0.2            # the 32-bit types serve small models
    dtype = "f32" if small else "bf16"
    kv_heads = rng.choice([1, 2, 4, 6, 8, 12, 16])
    heads = kv_heads * rng.choice([1, 1, 1, 2, 4])
    dim = rng.choice([16, 32, 40, 64, 64, 80, 96, 128, 128])
    train = rng.random() < 0.6
    if rng.random() < 0.25:
        # no more values than 8192 tokens of the largest listed case have
        tokens = _log_int(rng, 1, 600 if small else min(16384, 8192 * 40 * 128 // ((heads + kv_heads) * dim)))
        batch = rng.choice([b for b in (1, 2, 3, 8) if b <= tokens])
        interleaved = rng.random() < 0.3
        rot = dim if rng.random() < 0.6 else max(2, dim // 4 // 2 * 2)
        return {"op": "qk", "dtype": dtype, "batch": batch, "seq": max(1, tokens // batch),
                "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot, "train": train,
                "interleaved": interleaved}
    biased = rng.random() < 0.5
    causal = biased and rng.random() < 0.5
    batch = _log_int(rng, 1, 32)
    # scores of one head of one sequence: no more than 2^36 products of a query and a key
    # (f32: 2^30) and 2^29 scores over the batch; no more than 10^8 values of k
    most = min((1 << (30 if small else 36)) // (batch * heads * dim), (1 << 29) // (batch * heads))
    most_k = min(most, 10 ** 8 // (batch * kv_heads * dim), 300 if small else 32768)
    if not train and rng.random() < 0.4:       # the next token
        q_len, k_len = 1, _log_int(rng, 1, most_k)
    elif biased:                               # one sequence with itself
        q_len = k_len = _log_int(rng, 1, min(math.isqrt(most), most_k, 4096))
    else:
        k_len = _log_int(rng, 1, min(most_k, 16384))
        q_len = _log_int(rng, 1, max(1, min(most // k_len, 4096)))
    return {"op": "attn", "dtype": dtype, "batch": batch, "q_len": q_len, "k_len": k_len,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "train": train,
            "ragged": rng.random() < 0.6, "causal": causal,
            "buckets": rng.choice([16, 32, 64]) if biased else 0,
            "max_distance": rng.choice([64, 128, 250]) if biased else 128}


def _lens(case):
    """Keys of each sequence: spread evenly over (0, k_len], the last of eight or more empty
    (a batch filled up with an empty sequence)."""
    B, S = case["batch"], case["k_len"]
    if not case["ragged"]:
        return [S] * B
    lens = [max(1, math.ceil(S * ((0.5 + 0.6180339887 * (b + 1)) % 1.0))) for b in range(B)]
    if B >= 8:
        lens[-1] = 0
    return lens


def _starts(case):
    """Position of each sequence's first query: the last key's for a next token, else 0."""
    return [max(0, n - 1) if case["causal"] and case["q_len"] == 1 else 0 for n in _lens(case)]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    t = DTYPES[case["dtype"]]
    B, H, G, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]

    def normal(*shape, std=1.0, mean=0.0):
        v = torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)
        return v.mul_(std).add_(mean).to(t)

    state = {"case": case}
    if case["op"] == "qk":
        S, R = case["seq"], case["rot"]
        # the projection's output, heads of queries, keys and values side by side
        qkv = normal(B, S, H + 2 * G, D)
        state["q"], state["k"] = qkv[:, :, :H], qkv[:, :, H:H + G]
        state["wq"], state["wk"] = normal(D, std=0.1, mean=1.0), normal(D, std=0.1, mean=1.0)
        P = 32768                 # positions the model's tables hold
        angle = torch.arange(P, device="cuda", dtype=torch.float64)[:, None] * \
            10000.0 ** (-torch.arange(0, R, 2, device="cuda", dtype=torch.float64) / R)
        state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
        if S == 1:                # next tokens: each sequence at its own position
            state["positions"] = torch.randint(P, (B, 1), generator=gen, device="cuda")
        else:
            state["positions"] = None
        if case["train"]:
            state["dq"], state["dk"] = normal(B, S, H, D), normal(B, S, G, D)
        return state
    Sq, Sk = case["q_len"], case["k_len"]
    # scores of standard deviation near 1, with and without the factor of the plain form
    state["scale"] = 1.0 if case["buckets"] else D ** -0.5
    std = D ** -0.5 if case["buckets"] else 1.0
    if case["buckets"] and Sq == Sk:      # one projection of the sequence
        qkv = normal(B, Sk, H + 2 * G, D)
        qkv[:, :, :H] *= std
        state["q"], kv = qkv[:, :, :H], qkv[:, :, H:]
    else:                                 # queries of one sequence, keys and values of the other
        state["q"], kv = normal(B, Sq, H, D, std=std), normal(B, Sk, 2 * G, D)
    state["k"], state["v"] = kv[:, :, :G], kv[:, :, G:]
    ints = lambda v: torch.tensor(v, device="cuda", dtype=torch.int32)  # noqa: E731
    state["kv_lens"] = ints(_lens(case)) if case["ragged"] else None
    state["q_start"] = ints(_starts(case)) if any(_starts(case)) else None
    state["bias"] = normal(case["buckets"], H) if case["buckets"] else None
    if case["train"]:
        state["do"] = normal(B, Sq, H, D)
    return state


def _pairs(case):
    """Scores that count, over the batch, for one head."""
    n, S = 0, case["q_len"]
    for length, start in zip(_lens(case), _starts(case)):
        if not case["causal"]:
            n += S * length
            continue
        whole = min(S, max(0, start + S - length))       # queries that see every key
        n += whole * length + sum(min(length, start + i + 1) for i in range(S - whole))
    return n


def work(case):
    e = 4 if case["dtype"] == "f32" else 2
    B, H, G, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "qk":
        n, R = B * case["seq"] * (H + G) * D, case["rot"]
        tables = 4 * min(32768, B * case["seq"] if case["seq"] == 1 else case["seq"]) * R
        return {"bytes": e * n * (5 if case["train"] else 2) + tables,
                "flops": 8.0 * n * (3 if case["train"] else 1)}
    q, kv = B * case["q_len"] * H * D, sum(_lens(case)) * G * D
    lse = 4 * B * H * case["q_len"]
    n = e * (2 * q + 2 * kv) + lse + e * case["buckets"] * H
    if case["train"]:             # do, dq, dk, dv (dk and dv whole)
        n += e * (2 * q + 2 * B * case["k_len"] * G * D) + e * case["buckets"] * H
    return {"bytes": n, "flops": (14.0 if case["train"] else 4.0) * _pairs(case) * H * D}


# ---- the framework's operators ------------------------------------------------
def _run_own(s):
    from tensor_model_transformer_tp_gb300 import functional as F

    c = s["case"]
    if c["op"] == "qk":
        opt = {"positions": s["positions"], "q_weight": s["wq"], "k_weight": s["wk"], "eps": EPS,
               "interleaved": c["interleaved"]}
        q, k = F.qk_norm_rope_fwd(s["q"], s["k"], s["cos"], s["sin"], **opt)
        if not c["train"]:
            return {"q": q, "k": k}
        dq, dk, dwq, dwk = F.qk_norm_rope_bwd(s["q"], s["k"], s["dq"], s["dk"], s["cos"], s["sin"],
                                              **opt)
        return {"q": q, "k": k, "dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    opt = {"kv_lens": s["kv_lens"], "causal": c["causal"], "q_start": s["q_start"],
           "scale": s["scale"], "bias": s["bias"], "max_distance": c["max_distance"],
           "bidirectional": not c["causal"]}
    o, lse = F.attn_fwd(s["q"], s["k"], s["v"], **opt)
    if not c["train"]:
        return {"o": o, "lse": lse}
    dq, dk, dv, dbias = F.attn_bwd(s["q"], s["k"], s["v"], o, lse, s["do"], **opt)
    out = {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}
    return out | {"dbias": dbias} if c["buckets"] else out


# ---- the plain form -------------------------------------------------------------
def _borders(buckets, max_distance, bidirectional):
    """The smallest distance of every bucket but the first, for one sign."""
    n = buckets // 2 if bidirectional else buckets
    e = n // 2
    log = [e * (max_distance / e) ** (u / (n - e)) for u in range(1, n - e)]
    return list(range(1, e + 1)) + [math.ceil(x * (1 - 1e-12)) for x in log]


def _buckets(n, case):
    """bucket(n) of a tensor of relative positions."""
    both = not case["causal"]
    a = n.abs() if both else (-n).clamp_min(0)
    at = torch.tensor(_borders(case["buckets"], case["max_distance"], both), device=n.device)
    b = torch.bucketize(a, at, right=True)
    return torch.where(n > 0, b + case["buckets"] // 2, b) if both else b


def _turn(x, cos, sin, interleaved, back=False):
    """The rotation of the first values of x [B, S, heads, D] (its transpose where back)."""
    R = 2 * cos.shape[-1]
    c, s = cos[:, :, None], -sin[:, :, None] if back else sin[:, :, None]
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        turned = torch.stack([a * c - b * s, a * s + b * c], dim=-1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        turned = torch.cat([a * c - b * s, a * s + b * c], dim=-1)
    return torch.cat([turned, x[..., R:]], dim=-1)


def _norm_back(x, g, w):
    """Gradients of x and w behind the normalisation, g that of its output."""
    r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
    xh, gw = x * r, g * w
    dx = r * (gw - xh * (gw * xh).mean(dim=-1, keepdim=True))
    return dx, (g * xh).double().sum(dim=(0, 1, 2))


def _run_qk(s, t):
    c = s["case"]
    at = s["positions"]
    if at is None:
        at = torch.arange(c["seq"], device=s["q"].device)[None].expand(c["batch"], -1)
    cos, sin, il = s["cos"][at], s["sin"][at], c["interleaved"]

    def forward(x, w):
        x = x.float()
        r = torch.rsqrt(x.square().mean(dim=-1, keepdim=True) + EPS)
        return _turn(x * r * w.float(), cos, sin, il).to(t)

    out = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if not c["train"]:
        return out
    dq, dwq = _norm_back(s["q"].float(), _turn(s["dq"].float(), cos, sin, il, True), s["wq"].float())
    dk, dwk = _norm_back(s["k"].float(), _turn(s["dk"].float(), cos, sin, il, True), s["wk"].float())
    return out | {"dq": dq.to(t), "dk": dk.to(t), "dwq": dwq.to(t), "dwk": dwk.to(t)}


def _distances(s):
    """n = j - (q_start + i), [B or 1, Sq, Sk]."""
    c, dev = s["case"], s["q"].device
    i = torch.arange(c["q_len"], device=dev)[None, :, None]
    if s["q_start"] is not None:
        i = i + s["q_start"].long()[:, None, None]
    return torch.arange(c["k_len"], device=dev)[None, None] - i


def _visible(s):
    """Which keys count, [B or 1, 1, Sq or 1, Sk]; None: all."""
    c, see = s["case"], None
    if s["kv_lens"] is not None:
        keys = torch.arange(c["k_len"], device=s["q"].device)
        see = (keys[None] < s["kv_lens"][:, None])[:, None]
    if c["causal"]:
        past = _distances(s) <= 0
        see = past if see is None else see & past
    return None if see is None else see[:, None]


def _run_attn(s, t):
    c = s["case"]
    B, H, G, Sq, Sk = c["batch"], c["heads"], c["kv_heads"], c["q_len"], c["k_len"]
    # [B, key heads, query heads of each, tokens, D]
    q = s["q"].float().view(B, Sq, G, H // G, -1).permute(0, 2, 3, 1, 4)
    k, v = (s[x].float().permute(0, 2, 1, 3)[:, :, None] for x in "kv")
    score = (q @ k.transpose(-1, -2)).mul_(s["scale"]).view(B, H, Sq, Sk)
    if c["buckets"]:
        near = _buckets(_distances(s), c)
        score += s["bias"].float()[near].permute(0, 3, 1, 2)
    see = _visible(s)
    if see is not None:
        score = score.masked_fill_(~see, -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    top = torch.where(torch.isneginf(top), torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(dim=-1, keepdim=True)
    lse = (top + torch.log(total))[..., 0]
    p = p.div_(torch.where(total > 0, total, torch.ones_like(total))).view(B, G, H // G, Sq, Sk)
    o = (p @ v).permute(0, 3, 1, 2, 4).reshape(B, Sq, H, -1)
    out = {"o": o.to(t), "lse": lse}
    if not c["train"]:
        return out
    do = s["do"].float().view(B, Sq, G, H // G, -1).permute(0, 2, 3, 1, 4)
    dv = (p.transpose(-1, -2) @ do).sum(dim=2)
    dp = do @ v.transpose(-1, -2)
    ds = dp.sub_((p * dp).sum(dim=-1, keepdim=True)).mul_(p)
    dq = (ds @ k).mul_(s["scale"]).permute(0, 3, 1, 2, 4).reshape(B, Sq, H, -1)
    dk = (ds.transpose(-1, -2) @ q).sum(dim=2).mul_(s["scale"])
    out |= {"dq": dq.to(t), "dk": dk.permute(0, 2, 1, 3).to(t), "dv": dv.permute(0, 2, 1, 3).to(t)}
    if not c["buckets"]:
        return out
    # sums along the diagonals (rows turned round and shifted by one each), then by bucket
    W = Sq + Sk - 1
    skew = torch.nn.functional.pad(ds.reshape(B, H, Sq, Sk).flip(2), (0, Sq)).flatten(2)
    diagonal = skew[..., :Sq * W].view(B, H, Sq, W).sum(dim=2, dtype=torch.float64)
    n = torch.arange(W, device=ds.device)[None] - (Sq - 1)
    if s["q_start"] is not None:
        n = n - s["q_start"].long()[:, None]
    at = _buckets(n, c)[:, None].expand(B, H, W)
    dbias = torch.zeros(B, H, c["buckets"], device=ds.device, dtype=torch.float64)
    return out | {"dbias": dbias.scatter_add_(2, at, diagonal).sum(dim=0).t().to(t)}


def run(state):
    if own:
        return _run_own(state)
    t = DTYPES[state["case"]["dtype"]]
    return _run_qk(state, t) if state["case"]["op"] == "qk" else _run_attn(state, t)


# ---- the definition in 64 bits ----------------------------------------------------
def _bucket_of(n, buckets, max_distance, both):
    """bucket(n) of a whole number, the logarithm's floor decided by whole powers."""
    N = buckets // 2 if both else buckets
    a, base = (abs(n), N if n > 0 else 0) if both else (max(-n, 0), 0)
    E = N // 2
    if a < E:
        return base + a
    u = 0        # the largest u with (max_distance / E)^u <= (a / E)^(N - E)
    while u + 1 < N - E and max_distance ** (u + 1) * E ** (N - E) <= a ** (N - E) * E ** (u + 1):
        u += 1
    return base + E + u


def _exact_qk(s):
    c = s["case"]
    R, t = c["rot"], torch.float64
    at = s["positions"]
    if at is None:
        at = torch.arange(c["seq"], device="cuda").repeat(c["batch"], 1)
    turn = torch.complex(s["cos"][at].to(t), s["sin"][at].to(t))[:, :, None]

    def forward(x, w):
        y = torch.nn.functional.normalize(x, dim=-1, eps=0.0)      # x / |x|; eps beside it below
        size = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        y = y * (size / torch.sqrt(size ** 2 / c["dim"] + EPS)) * w
        if c["interleaved"]:
            pair = torch.view_as_complex(y[..., :R].unflatten(-1, (-1, 2)).contiguous())
            front = torch.view_as_real(pair * turn).flatten(-2)
        else:
            pair = torch.complex(y[..., :R // 2], y[..., R // 2:R]) * turn
            front = torch.cat([pair.real, pair.imag], dim=-1)
        return torch.cat([front, y[..., R:]], dim=-1)

    wide = [s[n].to(t).requires_grad_(True) for n in ("q", "k", "wq", "wk")]
    q, k = forward(wide[0], wide[2]), forward(wide[1], wide[3])
    out = {"q": q.detach(), "k": k.detach()}
    if c["train"]:
        got = torch.autograd.grad([q, k], wide, [s["dq"].to(t), s["dk"].to(t)])
        out |= dict(zip(("dq", "dk", "dwq", "dwk"), got))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk":
        return _exact_qk(s)
    t, c = torch.float64, case
    names = ["q", "k", "v"] + (["bias"] if c["buckets"] else [])
    wide = {n: s[n].to(t).requires_grad_(c["train"]) for n in names}
    share = c["heads"] // c["kv_heads"]
    k, v = (wide[n].repeat_interleave(share, dim=2) for n in "kv")
    score = torch.einsum("bihd,bjhd->bhij", wide["q"], k) * s["scale"]
    i = torch.arange(c["q_len"], device="cuda")[None] + torch.tensor(_starts(c), device="cuda")[:, None]
    n = torch.arange(c["k_len"], device="cuda")[None, None] - i[:, :, None]       # [B, Sq, Sk]
    if c["buckets"]:
        low, high = int(n.min()), int(n.max())
        known = torch.tensor([_bucket_of(x, c["buckets"], c["max_distance"], not c["causal"])
                              for x in range(low, high + 1)], device="cuda")
        # one product with the buckets' indicators for each distinct first position
        score = score + torch.nn.functional.embedding(known[n - low], wide["bias"]).permute(0, 3, 1, 2)
    hide = torch.arange(c["k_len"], device="cuda")[None, None] >= \
        torch.tensor(_lens(c), device="cuda")[:, None, None]
    if c["causal"]:
        hide = hide | (n > 0)
    hide = hide.expand(c["batch"], c["q_len"], c["k_len"])[:, None]
    none = hide.all(dim=-1, keepdim=True)
    lse = torch.logsumexp(score.masked_fill(hide, -math.inf).masked_fill(none, 0.0), dim=-1)
    weight = torch.softmax(score.masked_fill(hide, -math.inf).masked_fill(none, 0.0), dim=-1)
    o = torch.einsum("bhij,bjhd->bihd", weight.masked_fill(none, 0.0), v)
    out = {"o": o.detach(), "lse": lse.detach().masked_fill(none[..., 0], -math.inf)}
    if c["train"]:
        got = torch.autograd.grad(o, [wide[n] for n in names], s["do"].to(t))
        out |= dict(zip(["d" + n for n in names], got))
    return out
