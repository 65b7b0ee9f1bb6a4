"""The gated feed-forward block (oases_glu.h) and the linear head's cross entropy
(oases_ce.h) on the GPU, against float64 definitions (oracle/glu.py,
oracle/head.py), element by element.

Bounds.  u = 2^-8 (bf16) or 2^-24 (fp32) is half a step of the storage type
relative to the value.  A product over K terms accumulated in fp32, in any
order and truncated or rounded, is off by at most K 2^-23 sum |terms| (g_K
below).  The element-wise functions (hardware exponential and reciprocal, the
7.1.26 rational form of erf with absolute error 1.5e-7) are given EW = 2^-19
relative to |a b|, |dh b| and so on, which act and act' stay below 1.13 of.
Each bound is the first-order propagation of those three through the formulas
with a factor 1.05 for the products of errors; nothing is fitted.
"""
import numpy as np
import pytest
import torch

import oracle.fp8 as fp8
import tensor_model_transformer_tp_gb300 as oz
from oracle.glu import act_and_grad, glu_backward, glu_output, glu_projections
from oracle.head import ce_backward, ce_forward
from tensor_model_transformer_tp_gb300 import functional as F

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EW = 2.0 ** -19
D1 = 1.13      # max |act'| (1.0998 SiLU, 1.129 GeLU)
D2 = 0.80      # max |act''| (0.5 SiLU, 0.798 GeLU)
SLACK = 1.05


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def g_(K):
    return K * 2.0 ** -23


def f64(t):
    return t.detach().double().cpu().numpy()


def inside(got, want, bound, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    bad = ~(np.abs(got - want) <= SLACK * bound + 1e-30)
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the bound, first at %s (%r, want %r)" % (
        what, bad.sum(), bad.size, np.nanmax(np.abs(got - want) / (bound + 1e-30)),
        np.argwhere(bad)[0], got[tuple(np.argwhere(bad)[0])], want[tuple(np.argwhere(bad)[0])])


def glu_case(dtype, M, H, Fn, bias, resid, seed=0):
    gen = torch.Generator().manual_seed(1000 * seed + M + 7 * H + 13 * Fn)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(T[dtype]).cuda()

    w = {"w1": rnd(2 * Fn, H, std=H ** -0.5), "w2": rnd(H, Fn, std=Fn ** -0.5)}
    if bias:
        w |= {"b1": rnd(2 * Fn, std=0.5), "b2": rnd(H, std=0.5)}
    return rnd(M, H), w, rnd(M, H) if resid else None, rnd(M, H)


def projection_bounds(x, w, a, b):
    """How far a and b in fp32 may be off."""
    H, Fn = x.shape[1], a.shape[1]
    e = g_(H) * (np.abs(x) @ np.abs(w["w1"]).T)
    if w.get("b1") is not None:
        e = e + 2.0 ** -23 * (np.abs(np.concatenate([a, b], axis=1)) + np.abs(w["b1"]))
    return e[:, :Fn], e[:, Fn:]


def kept_values(saved, save, M, Fn):
    """(a, b) float64 as the backward reads them."""
    if save == "pre":
        v = f64(saved)
        return v[:, :Fn], v[:, Fn:]
    ldq = (Fn + 15) // 16 * 16
    raw = saved.cpu().numpy()
    codes = raw[:2 * M * ldq].reshape(2, M, ldq)[:, :, :Fn]
    at = (2 * M * ldq + 255) // 256 * 256
    kg = (Fn + 127) // 128
    n = (M + 127) // 128 * kg * 512
    sc = raw[at:at + 2 * n].reshape(2, n).astype(np.int64)
    r, j = np.arange(M)[:, None], (np.arange(Fn) // 32)[None, :]
    off = ((r // 128) * kg + j // 4) * 512 + (r % 32) * 16 + ((r % 128) // 32) * 4 + j % 4
    vals = fp8.e4m3_decode(np.arange(256))
    return tuple(vals[codes[k]] * 2.0 ** (sc[k][off] - 127.0) for k in (0, 1))


def check_kept(saved, save, dtype, a, b, ea, eb):
    M, Fn = a.shape
    for got, want, err, what in zip(kept_values(saved, save, M, Fn), (a, b), (ea, eb), "ab"):
        if save == "pre":
            inside(got, want, U[dtype] * np.abs(want) + err, "kept " + what)
            continue
        # 8 bits: X = 2^(floor log2 max - 8) of each 32 columns, the nearest
        # E4M3 value of v / X; where max |v| is within the fp32 error of a power
        # of two either scale may be taken, and saturation at 448 X cuts up to 1/8
        for j in range(0, Fn, 32):
            v, d, g = want[:, j:j + 32], err[:, j:j + 32], got[:, j:j + 32]
            top, slip = np.abs(v).max(axis=1, keepdims=True), d.max(axis=1, keepdims=True)
            ok = np.zeros(v.shape, bool)
            for t in (top - slip, top + slip):
                X = 2.0 ** (np.floor(np.log2(np.maximum(t, 2.0 ** -100))) - 8)
                r = np.clip(v / X, -448, 448)
                half = np.maximum(2.0 ** (np.floor(np.log2(np.maximum(np.abs(r), 2.0 ** -6))) - 4),
                                  2.0 ** -10)
                ok |= np.abs(g / X - r) <= half * (1 + 1e-9) + d / X
            assert ok.all(), ("kept " + what, j, np.argwhere(~ok)[:3])


GLU_SHAPES = [
    ("bf16", 1, 64, 104), ("bf16", 2, 2560, 512), ("bf16", 7, 72, 136), ("bf16", 33, 520, 264),
    ("bf16", 128, 256, 512), ("bf16", 129, 264, 520), ("bf16", 300, 512, 1000),
    ("bf16", 257, 128, 2048), ("bf16", 640, 1032, 776), ("bf16", 1, 8, 8),
    ("bf16", 17, 1096, 72), ("bf16", 65, 264, 1160), ("bf16", 180, 200, 3000),
    ("f32", 1, 33, 17), ("f32", 5, 64, 100), ("f32", 130, 97, 250), ("f32", 200, 256, 520),
    ("f32", 1, 1, 1),
]
GLU_OPTIONS = [("silu", "none", True, True), ("gelu", "pre", False, False),
               ("silu", "mxfp8", True, False), ("gelu", "none", False, True),
               ("gelu", "mxfp8", False, True), ("silu", "pre", True, True)]


# (activations are kept in 8 bits beside bf16 storage only)
@pytest.mark.parametrize("dtype,M,H,Fn,act,save,bias,resid",
                         [s + o for s in GLU_SHAPES for o in GLU_OPTIONS
                          if s[0] == "bf16" or o[1] != "mxfp8"])
def test_glu_forward_and_backward(dtype, M, H, Fn, act, save, bias, resid):
    x, w, r, dy = glu_case(dtype, M, H, Fn, bias, resid)
    u = U[dtype]
    y, saved = F.glu_fwd(x, w, act=act, resid=r, save=save)
    dx, grads = F.glu_bwd(x, dy, w, act=act, save=save, saved=saved)
    oz.oases_check_device(torch.cuda.current_stream())
    X, W, DY = f64(x), {k: f64(v) for k, v in w.items()}, f64(dy)
    R = None if r is None else f64(r)
    a, b = glu_projections(X, W)
    ea, eb = projection_bounds(X, W, a, b)
    f, df = act_and_grad(a, act)
    h = f * b
    eh = D1 * ea * np.abs(b) + np.abs(f) * eb + EW * np.abs(a * b) + u * np.abs(h)
    want = glu_output(a, b, W, act, R)
    ey = eh @ np.abs(W["w2"]).T + g_(Fn) * (np.abs(h) @ np.abs(W["w2"]).T) + u * np.abs(want)
    ey = ey + 2.0 ** -22 * (np.abs(want) + (np.abs(W["b2"]) if bias else 0)
                            + (np.abs(R) if resid else 0))
    inside(y, want, ey, "y")

    # the backward pass at the values it was given (or, computed again, at the
    # projections as they are)
    if save == "none":
        ka, kb, da_, db_ = a, b, ea, eb      # from the fp32 accumulators
    else:
        check_kept(saved, save, dtype, a, b, ea, eb)
        ka, kb = kept_values(saved, save, M, Fn)
        da_ = db_ = np.zeros_like(ka)
    f, df = act_and_grad(ka, act)
    dh = DY @ W["w2"]
    edh = g_(H) * (np.abs(DY) @ np.abs(W["w2"]))
    da, db = dh * kb * df, dh * f
    eda = (np.abs(kb * df) * edh + np.abs(dh) * (D1 * db_ + np.abs(kb) * D2 * da_)
           + EW * np.abs(dh * kb) + u * np.abs(da))
    edb = np.abs(f) * edh + np.abs(dh) * D1 * da_ + EW * np.abs(dh * ka) + u * np.abs(db)
    eh = D1 * da_ * np.abs(kb) + np.abs(f) * db_ + EW * np.abs(ka * kb) + u * np.abs(f * kb)
    dp, edp = np.concatenate([da, db], 1), np.concatenate([eda, edb], 1)
    wdx, wg = glu_backward(DY, X, ka, kb, W, act)
    A = np.abs
    inside(dx, wdx, edp @ A(W["w1"]) + g_(2 * Fn) * (A(dp) @ A(W["w1"])) + u * A(wdx), "dx")
    inside(grads["w1"], wg["w1"], edp.T @ A(X) + g_(M) * (A(dp).T @ A(X)) + u * A(wg["w1"]), "dw1")
    inside(grads["w2"], wg["w2"], A(DY).T @ eh + g_(M) * (A(DY).T @ A(f * kb)) + u * A(wg["w2"]),
           "dw2")
    assert set(grads) == set(w)
    if bias:
        inside(grads["b1"], wg["b1"], edp.sum(0) + g_(M) * A(dp).sum(0) + u * A(wg["b1"]), "db1")
        inside(grads["b2"], wg["b2"], g_(M) * A(DY).sum(0) + u * A(wg["b2"]), "db2")


@pytest.mark.parametrize("dtype,M,H,Fn", [("bf16", 140, 136, 264), ("f32", 9, 40, 50),
                                          ("bf16", 3, 512, 256), ("bf16", 5003, 72, 136)])
def test_glu_accumulated_fp32_gradients(dtype, M, H, Fn):
    """grads given: fp32, added to, the same sums as written gradients; a subset
    leaves the others out; dx as fp32."""
    x, w, _, dy = glu_case(dtype, M, H, Fn, True, False)
    start = {k: torch.randn_like(v, dtype=torch.float32) for k, v in w.items()}
    acc = {k: v.clone() for k, v in start.items()}
    dx, got = F.glu_bwd(x, dy, w, grads=acc, dx_dtype=torch.float32)
    dx_t, plain = F.glu_bwd(x, dy, w)
    assert got is acc and dx.dtype == torch.float32
    assert torch.equal(dx.to(dx_t.dtype), dx_t)
    for k in w:
        sums = acc[k].double() - start[k].double()
        # the addition rounds to fp32; the written form rounds to the storage type
        tol = 2.0 ** -23 * (start[k].abs() + acc[k].abs()).double() + U[dtype] * sums.abs() * 1.01
        assert ((plain[k].double() - sums).abs() <= tol + 1e-30).all(), k
    only = {"w2": torch.zeros_like(w["w2"], dtype=torch.float32)}
    dx2, _ = F.glu_bwd(x, dy, w, grads=only, need_dx=False)
    assert dx2 is None
    assert torch.equal(only["w2"].to(T[dtype]), plain["w2"])


def test_glu_residual_in_place_and_guard_bands():
    """y may be resid; nothing beside the outputs is written."""
    M, H, Fn = 131, 200, 328
    x, w, r, dy = glu_case("bf16", M, H, Fn, True, True)
    y, saved8 = F.glu_fwd(x, w, resid=r, save="mxfp8")
    band = 4096

    def guarded(nbytes):
        buf = torch.full((nbytes + 2 * band,), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, buf.data_ptr() + band

    def intact(buf):
        return bool((buf[:band] == 0xA5).all() and (buf[-band:] == 0xA5).all())

    for keep, name in ((0, "none"), (1, "pre"), (2, "mxfp8")):
        d = oz.GluDesc(1, M, H, Fn, 0, keep, 1, 1, 0)
        bufs = {"y": guarded(M * H * 2), "s": guarded(oz.oases_glu_saved_bytes(d)),
                "w": guarded(oz.oases_glu_workspace_bytes(d, False)),
                "v": guarded(oz.oases_glu_workspace_bytes(d, True)), "dx": guarded(M * H * 2)}
        gr = {k: guarded(v.numel() * 2) for k, v in w.items()}
        bufs["y"][0][band:-band] = r.view(torch.uint8).flatten()
        saved = bufs["s"][1] if keep else None
        oz.oases_glu_fwd(d, w, x, bufs["y"][1], bufs["y"][1], saved, bufs["w"][1],
                         oz.oases_glu_workspace_bytes(d, False))
        oz.oases_glu_bwd(d, w, x, dy, saved, bufs["dx"][1], {k: v[1] for k, v in gr.items()},
                         bufs["v"][1], oz.oases_glu_workspace_bytes(d, True))
        torch.cuda.synchronize()
        assert torch.equal(bufs["y"][0][band:-band].view(torch.bfloat16).view(M, H), y), name
        for k, (buf, _) in {**bufs, **gr}.items():
            assert intact(buf), (name, k)
        if keep == 2:
            ldq = (Fn + 15) // 16 * 16
            a = bufs["s"][0][band:-band].cpu().numpy()
            b = saved8.cpu().numpy()
            codes = lambda v: v[:2 * M * ldq].reshape(2, M, ldq)[:, :, :Fn]  # noqa: E731
            np.testing.assert_array_equal(codes(a), codes(b))
            at = (2 * M * ldq + 255) // 256 * 256
            np.testing.assert_array_equal(a[at:], b[at:])


def test_glu_kept_scales_past_the_matrix_hold_one():
    M, H, Fn = 37, 64, 72
    x, w, _, _ = glu_case("bf16", M, H, Fn, False, False)
    _, saved = F.glu_fwd(x, w, save="mxfp8")
    ldq, kg = 80, 1
    raw = saved.cpu().numpy()
    sc = raw[(2 * M * ldq + 255) // 256 * 256:].reshape(2, -1)
    assert sc.shape[1] == kg * 512
    used = np.zeros(512, bool)
    for r in range(M):
        for j in range(3):
            used[(r % 32) * 16 + (r // 32) * 4 + j] = True
    assert (sc[:, ~used] == 127).all()


def test_glu_extreme_and_non_finite_values_stay_in_their_rows():
    """Large gates saturate the activations; inf and NaN rows leave others alone."""
    M, H, Fn = 40, 64, 128
    x, w, _, dy = glu_case("bf16", M, H, Fn, False, False)
    x[3] *= 1e4
    x[4] = 0
    y0, s0 = F.glu_fwd(x, w, save="pre")
    x2 = x.clone()
    x2[7, 5] = float("nan")
    x2[8, 6] = float("inf")
    for act in ("silu", "gelu"):
        y0, _ = F.glu_fwd(x, w, act=act)
        y, _ = F.glu_fwd(x2, w, act=act)
        assert torch.isfinite(y0).all()
        assert y[7].isnan().all() and not torch.isfinite(y[8]).all()
        keep = [m for m in range(M) if m not in (7, 8)]
        assert torch.equal(y[keep], y0[keep])
        dx0, _ = F.glu_bwd(x, dy, w, act=act)
        dx, _ = F.glu_bwd(x2, dy, w, act=act)
        assert torch.equal(dx[keep], dx0[keep]) and dx[7].isnan().all()


CE_SHAPES = [
    ("bf16", 1, 64, 1), ("bf16", 1, 1024, 3001), ("bf16", 5, 72, 2), ("bf16", 37, 264, 1003),
    ("bf16", 128, 128, 256), ("bf16", 130, 520, 5000), ("bf16", 300, 64, 777),
    ("bf16", 513, 256, 12289), ("bf16", 2, 8, 40000),
    ("f32", 1, 17, 33), ("f32", 9, 64, 1003), ("f32", 130, 97, 400), ("f32", 3, 5, 1),
]


def ce_case(dtype, M, H, V, per_row, seed=0, std=1.0):
    gen = torch.Generator().manual_seed(100 * seed + M + 3 * H + 5 * V)
    x = torch.randn(M, H, generator=gen).to(T[dtype]).cuda()
    w = (torch.randn(V, H, generator=gen) * std * H ** -0.5).to(T[dtype]).cuda()
    t = torch.randint(0, V, (M,), generator=gen)
    if M > 2:
        t[1], t[2] = -100, V - 1
    d = torch.rand(M if per_row else 1, generator=gen) / M - (0.3 / M if per_row else 0)
    return x, w, t.cuda(), d.cuda()


def ce_bounds(x, w, t):
    """(loss, lse, logits, error of the logits, of lse, of loss)."""
    loss, lse, l = ce_forward(x, w, t)
    el = g_(x.shape[1]) * (np.abs(x) @ np.abs(w).T)
    elog = el.max(axis=1) + 2.0 ** -18 + 2.0 ** -22 * np.abs(lse)
    used = t != -100
    at = np.where(used, t, 0)
    eloss = np.where(used, elog + el[np.arange(len(t)), at] + 2.0 ** -23 * np.abs(loss), 0.0)
    return loss, lse, l, el, elog, eloss


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("dtype,M,H,V", CE_SHAPES)
def test_ce_forward_and_backward(dtype, M, H, V, per_row):
    x, w, t, d = ce_case(dtype, M, H, V, per_row, std=2.0)
    loss, lse = F.ce_fwd(x, w, t)
    dx, dw = F.ce_bwd(x, w, t, lse, d)
    oz.oases_check_device(torch.cuda.current_stream())
    X, W, tt = f64(x), f64(w), t.cpu().numpy()
    D = np.broadcast_to(f64(d), (M,))
    wl, wlse, l, el, elog, eloss = ce_bounds(X, W, tt)
    inside(lse, wlse, elog, "lse")
    inside(loss, wl, eloss, "loss")
    wdx, wdw, g = ce_backward(X, W, tt, D)
    u = U[dtype]
    p = np.exp(l - wlse[:, None])
    used = (tt != -100)[:, None]
    eg = np.where(used, np.abs(D)[:, None] * p * (el + elog[:, None] + 2.0 ** -18)
                  + (u + 2.0 ** -22) * np.abs(g) + 2.0 ** -24 * np.abs(D)[:, None] * p, 0.0)
    A = np.abs
    inside(dx, wdx, eg @ A(W) + g_(V) * (A(g) @ A(W)) + u * A(wdx), "dx")
    inside(dw, wdw, eg.T @ A(X) + g_(M) * (A(g).T @ A(X)) + u * A(wdw), "dw")
    if M > 2:
        assert loss[1] == 0 and not dx[1].any()


@pytest.mark.parametrize("dtype,M,H,V", [("bf16", 70, 136, 900), ("f32", 11, 30, 100),
                                         ("bf16", 5003, 72, 300)])
def test_ce_accumulated_fp32_gradient(dtype, M, H, V):
    x, w, t, d = ce_case(dtype, M, H, V, True)
    _, lse = F.ce_fwd(x, w, t)
    dx, dw = F.ce_bwd(x, w, t, lse, d)
    start = torch.randn_like(dw, dtype=torch.float32)
    acc = start.clone()
    dx2, got = F.ce_bwd(x, w, t, lse, d, dw=acc)
    assert got is acc and torch.equal(dx, dx2)
    sums = acc.double() - start.double()
    tol = 2.0 ** -23 * (start.abs() + acc.abs()).double() + U[dtype] * 1.01 * sums.abs()
    assert ((dw.double() - sums).abs() <= tol + 1e-30).all()
    only_dx, none = F.ce_bwd(x, w, t, lse, d, need_dw=False)
    assert none is None and torch.equal(only_dx, dx)
    none, only_dw = F.ce_bwd(x, w, t, lse, d, need_dx=False)
    assert none is None and torch.equal(only_dw, dw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_ce_gradient_against_differences_of_the_loss(dtype):
    """d sum(loss dloss) along random directions of x: the loss of the kernel
    itself at x + e and x - e (powers of two apart, exact in the storage type)."""
    M, H, V = 6, 64, 300
    x, w, t, d = ce_case(dtype, M, H, V, True)
    x = torch.round(x.float() * 8).clamp(-15, 15).div(8).to(T[dtype])    # room for +- 1/16 in bf16
    _, lse = F.ce_fwd(x, w, t)
    dx, _ = F.ce_bwd(x, w, t, lse, d)
    step = 2.0 ** -4
    gen = torch.Generator().manual_seed(5)
    for _ in range(4):
        v = (torch.randint(0, 2, (M, H), generator=gen) * 2 - 1).cuda().float()
        up, dn = (x.float() + step * v), (x.float() - step * v)
        assert torch.equal(up.to(T[dtype]).float(), up)
        lu, ld = (F.ce_fwd(q.to(T[dtype]), w, t)[0].double() for q in (up, dn))
        for m in range(M):
            num = float((lu[m] - ld[m]) * d[m].double()) / (2 * step)
            ana = float((dx[m].double() * v[m].double()).sum())
            # third-order remainder: |phi'''| <= max |w.v|^3 along the direction
            b = float((w.float() @ v[m]).abs().max())
            rem = abs(float(d[m])) * step ** 2 / 6 * (2 * b) ** 3
            rnd = U[dtype] * float(dx[m].double().abs().sum()) * 2 + abs(float(d[m])) * 2e-5 / step
            assert abs(num - ana) <= rem + rnd, (m, num, ana, rem, rnd)


def test_ce_bad_targets_give_nan_and_extreme_logits_do_not():
    x, w, t, d = ce_case("bf16", 20, 64, 500, False)
    loss0, lse0 = F.ce_fwd(x, w, t)
    t2 = t.clone()
    t2[5], t2[6] = 500, -7
    loss, lse = F.ce_fwd(x, w, t2)
    assert torch.equal(lse, lse0)
    assert loss[5].isnan() and loss[6].isnan()
    rest = [m for m in range(20) if m not in (5, 6)]
    assert torch.equal(loss[rest], loss0[rest])
    dx0, _ = F.ce_bwd(x, w, t, lse0, d)
    dx, dw = F.ce_bwd(x, w, t2, lse, d)
    assert dx[5].isnan().all() and dw.isnan().all()
    assert torch.equal(dx[rest], dx0[rest])
    # logits in the thousands: no overflow, probabilities 0 and 1
    big = x * 300
    loss, lse = F.ce_fwd(big, w, t)
    wl, wlse, _, _, elog, eloss = ce_bounds(f64(big), f64(w), t.cpu().numpy())
    inside(lse, wlse, elog, "lse")
    inside(loss, wl, eloss, "loss")
    dx, dw = F.ce_bwd(big, w, t, lse, d)
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()


def test_ce_ignored_rows_count_for_nothing_whatever_they_hold():
    x, w, t, d = ce_case("bf16", 12, 64, 300, False)
    t[4] = -100
    x2 = x.clone()
    x2[4] = float("nan")
    loss, lse = F.ce_fwd(x2, w, t)
    assert loss[4] == 0
    dx, dw = F.ce_bwd(x2, w, t, lse, d)
    assert not dx[4].any()
    # every row ignored: all zero
    t[:] = 7
    loss, lse = F.ce_fwd(x, w, t, ignore_index=7)
    dx, dw = F.ce_bwd(x, w, t, lse, d, ignore_index=7)
    assert not loss.any() and not dx.any() and not dw.any()


def test_ce_targets_may_be_a_slice_and_dloss_infinite():
    """Shifted targets start 8 bytes into their buffer; an infinite dloss of one
    row stays in that row's dx."""
    x, w, t, d = ce_case("bf16", 12, 64, 300, True)
    tokens = torch.cat([t[:1], t])
    loss0, lse0 = F.ce_fwd(x, w, t)
    loss, lse = F.ce_fwd(x, w, tokens[1:])
    assert torch.equal(loss, loss0) and torch.equal(lse, lse0)
    dx0, _ = F.ce_bwd(x, w, t, lse0, d)
    d2 = d.clone()
    d2[3] = float("inf")
    d2[1] = float("nan")        # an ignored row
    dx, _ = F.ce_bwd(x, w, tokens[1:], lse0, d2)
    rest = [m for m in range(12) if m != 3]
    assert not torch.isfinite(dx[3]).any()
    # the common factor is another one without row 3: one bf16 step at most
    assert ((dx[rest].double() - dx0[rest].double()).abs()
            <= 2.0 ** -6 * dx0[rest].double().abs().amax(dim=1, keepdim=True)).all()


def test_ce_minus_infinity_logits():
    """A vocabulary entry masked by -inf weights (x > 0): probability 0."""
    gen = torch.Generator().manual_seed(3)
    M, H, V = 9, 64, 700
    x = (torch.rand(M, H, generator=gen) + 0.5).to(torch.bfloat16).cuda()
    w = (torch.randn(V, H, generator=gen) * 0.1).to(torch.bfloat16).cuda()
    t = torch.randint(0, 256, (M,), generator=gen).cuda()
    loss0, lse0 = F.ce_fwd(x, w[:256].contiguous(), t)
    w[256:] = float("-inf")
    loss, lse = F.ce_fwd(x, w, t)
    assert torch.isfinite(loss).all()
    assert (lse - lse0).abs().max() <= 2.0 ** -18 and (loss - loss0).abs().max() <= 2.0 ** -18


def _rms_close(got, want, rel, what):
    """Relative 2-norm, for sizes whose element-wise bounds would take minutes."""
    r = float((got.double() - want).norm() / want.norm())
    assert r <= rel, (what, r)


@pytest.mark.parametrize("M,H,Fn,save", [(4096, 1024, 6000, "mxfp8"), (3000, 2048, 5464, "pre"),
                                         (8200, 512, 1032, "none"), (40000, 264, 520, "pre"),
                                         (12001, 256, 136, "mxfp8")])
def test_glu_larger_sizes(M, H, Fn, save):
    """Products that take several launches or share one, on float64 products of
    the same roundings' size: kept and intermediate values carry up to three bf16
    roundings of 2^-9 rms each and the output one more, 2 * 2^-9 in all."""
    x, w, r, dy = glu_case("bf16", M, H, Fn, True, True)
    y, saved = F.glu_fwd(x, w, resid=r, save=save)
    dx, grads = F.glu_bwd(x, dy, w, save=save, saved=saved)
    oz.oases_check_device(torch.cuda.current_stream())
    W = {k: v.double() for k, v in w.items()}
    p = x.double() @ W["w1"].t() + W["b1"]
    a, b = p[:, :Fn], p[:, Fn:]
    _rms_close(y, (a * torch.sigmoid(a) * b) @ W["w2"].t() + W["b2"] + r.double(), 2.0 ** -8, "y")
    if save != "none":
        a, b = (torch.from_numpy(v).cuda() for v in kept_values(saved, save, M, Fn))
    s = torch.sigmoid(a)
    dh = dy.double() @ W["w2"]
    dp = torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], dim=1)
    _rms_close(dx, dp @ W["w1"], 2.0 ** -8, "dx")
    _rms_close(grads["w1"], dp.t() @ x.double(), 2.0 ** -8, "dw1")
    _rms_close(grads["w2"], dy.double().t() @ (a * s * b), 2.0 ** -8, "dw2")
    _rms_close(grads["b1"], dp.sum(0), 2.0 ** -8, "db1")
    _rms_close(grads["b2"], dy.double().sum(0), 2.0 ** -8, "db2")


@pytest.mark.parametrize("M,H,V", [(8000, 256, 20001), (300, 512, 60000), (4096, 1024, 33000),
                                   (2000, 128, 100), (30001, 264, 1000), (40000, 72, 9000)])
def test_ce_larger_sizes(M, H, V):
    """Several pieces of the vocabulary (8000 x 20001 logits), split contractions
    and products that share a launch or do not."""
    x, w, t, d = ce_case("bf16", M, H, V, True, std=2.0)
    loss, lse = F.ce_fwd(x, w, t)
    dx, dw = F.ce_bwd(x, w, t, lse, d)
    oz.oases_check_device(torch.cuda.current_stream())
    l = x.double() @ w.double().t()
    ref = torch.logsumexp(l, dim=1)
    used = t != -100
    at = torch.where(used, t, 0)[:, None]
    want = torch.where(used, ref - l.gather(1, at)[:, 0], torch.zeros_like(ref))
    assert (lse.double() - ref).abs().max() <= 1e-5 * ref.abs().max()
    assert (loss.double() - want).abs().max() <= 1e-5 * want.abs().max()
    g = torch.exp(l - ref[:, None]).scatter_add_(1, at, -torch.ones_like(ref)[:, None])
    g = g * torch.where(used, d.double(), torch.zeros_like(ref))[:, None]
    _rms_close(dx, g @ w.double(), 2.0 ** -8, "dx")
    _rms_close(dw, g.t() @ x.double(), 2.0 ** -8, "dw")


@pytest.mark.parametrize("dtype,M,H,Fn", [("bf16", 1023, 8, 16), ("bf16", 1024, 16, 8), ("bf16", 2049, 72, 136),
                                          ("bf16", 9001, 8, 64), ("f32", 1030, 3, 5), ("f32", 4097, 9, 40),
                                          ("f32", 9001, 2, 2)])
def test_glu_bias_gradients_of_many_rows_are_exact(dtype, M, H, Fn):
    """Sums of small whole numbers, exact in any order: one row of w2 is not 0, so
    |dh| <= 1, and a = 32, where the exact GeLU is a and its derivative 1, so
    da = dh b and db = 32 dh."""
    gen = torch.Generator().manual_seed(M + H)

    def whole(lo, hi, *shape):
        return torch.randint(lo, hi + 1, shape, generator=gen).to(T[dtype]).cuda()

    x, dy = whole(-1, 1, M, H), whole(-1, 1, M, H)
    w2 = torch.zeros(H, Fn, dtype=T[dtype], device="cuda")
    w2[H - 1] = whole(-1, 1, Fn)
    w = {"w1": whole(-1, 1, 2 * Fn, H), "w2": w2, "b1": whole(0, 0, 2 * Fn), "b2": whole(0, 0, H)}
    b = whole(-3, 3, M, Fn)
    saved = torch.cat([torch.full_like(b, 32.0), b], dim=1)
    dh = dy[:, H - 1:].double() * w2[H - 1].double()
    db1 = torch.cat([dh * b.double(), 32 * dh], dim=1).sum(0)
    db2 = dy.double().sum(0)
    prior = {k: whole(-5, 5, *w[k].shape).float() for k in ("b1", "b2")}
    grads = {k: v.clone() for k, v in prior.items()}
    F.glu_bwd(x, dy, w, act="gelu", save="pre", saved=saved, grads=grads, need_dx=False)
    assert torch.equal(grads["b1"].double(), prior["b1"].double() + db1)
    assert torch.equal(grads["b2"].double(), prior["b2"].double() + db2)
    _, grads = F.glu_bwd(x, dy, w, act="gelu", save="pre", saved=saved)
    assert torch.equal(grads["b1"], db1.to(T[dtype])) and torch.equal(grads["b2"], db2.to(T[dtype]))


def test_empty_batches():
    for dtype in ("bf16", "f32"):
        x, w, _, dy = glu_case(dtype, 0, 64, 104, True, False)
        for save in ("none", "pre"):
            y, saved = F.glu_fwd(x, w, save=save)
            dx, grads = F.glu_bwd(x, dy, w, save=save, saved=saved)
            assert y.shape == dx.shape == (0, 64)
            assert all(not g.any() for g in grads.values())
        head = torch.randn(50, 64).to(T[dtype]).cuda()
        t = torch.zeros(0, dtype=torch.int64, device="cuda")
        loss, lse = F.ce_fwd(x, head, t)
        dx, dw = F.ce_bwd(x, head, t, lse, torch.ones(1, device="cuda"))
        assert loss.shape == (0,) and not dw.any() and dw.shape == head.shape


def _chain(x, w, head, t, d):
    """Feed-forward block with residual, then the head: (loss, dx, gradients)."""
    y, saved = F.glu_fwd(x, w, resid=x, save="pre")
    loss, lse = F.ce_fwd(y, head, t)
    dy, dhead = F.ce_bwd(y, head, t, lse, d)
    dx, grads = F.glu_bwd(x, dy, w, save="pre", saved=saved)
    return [loss, dx + dy, dhead] + [grads[k] for k in sorted(grads)]


@pytest.mark.parametrize("M", [5, 200])
def test_repeated_calls_other_streams_and_captured_graphs_give_the_same_bits(M):
    x, w, _, _ = glu_case("bf16", M, 256, 512, True, False)
    _, head, t, d = ce_case("bf16", M, 256, 1500, True)
    want = [v.clone() for v in _chain(x, w, head, t, d)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:          # three in flight at once, each with its own workspace
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(_chain(x, w, head, t, d))
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want):
            assert torch.equal(a, b)
    # two captured graphs, replayed with other inputs between
    xs = x.clone()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(_chain(xs, w, head, t, d))
        graphs.append(g)
    for g in graphs:
        xs.copy_(x.flip(0))
        g.replay()
    xs.copy_(x)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, want):
            assert torch.equal(a, b)
    oz.oases_check_device(torch.cuda.current_stream())


def test_two_host_threads_on_their_own_streams():
    import threading

    jobs = []
    for M in (5, 300):
        x, w, _, _ = glu_case("bf16", M, 256, 512, True, False)
        _, head, t, d = ce_case("bf16", M, 256, 1500, True)
        jobs.append((x, w, head, t, d, [v.clone() for v in _chain(x, w, head, t, d)]))
    torch.cuda.synchronize()
    wrong = []

    def work(x, w, head, t, d, want):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = _chain(x, w, head, t, d)
            torch.cuda.current_stream().synchronize()
        wrong.extend(i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work, args=j) for j in jobs]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not wrong
    oz.oases_check_device(None)


def test_refusals_of_torch_arguments():
    x, w, r, dy = glu_case("bf16", 4, 64, 128, True, True)
    head, t = torch.randn(30, 64).bfloat16().cuda(), torch.zeros(4, dtype=torch.int64).cuda()
    bad = [
        lambda: F.glu_fwd(x.t(), w), lambda: F.glu_fwd(x.half(), w), lambda: F.glu_fwd(x[None], w),
        lambda: F.glu_fwd(x, {**w, "w1": w["w1"].float()}),
        lambda: F.glu_fwd(x, {**w, "w1": w["w1"][:-1]}),
        lambda: F.glu_fwd(x, {**w, "w2": w["w2"].t()}), lambda: F.glu_fwd(x, {"w1": w["w1"]}),
        lambda: F.glu_fwd(x, {**w, "w3": w["w2"]}), lambda: F.glu_fwd(x, w, act="relu"),
        lambda: F.glu_fwd(x, w, save="fp8"), lambda: F.glu_fwd(x, w, resid=r[:2]),
        lambda: F.glu_fwd(x, {k: v.cpu() for k, v in w.items()}),
        lambda: F.glu_bwd(x, dy, w, save="pre"), lambda: F.glu_bwd(x, dy, w, saved=r),
        lambda: F.glu_bwd(x, dy[:2], w), lambda: F.glu_bwd(x, dy, w, grads={"w1": w["w1"]}),
        lambda: F.glu_bwd(x, dy, w, dx_dtype=torch.float16),
        lambda: F.glu_bwd(x, dy, {k: w[k] for k in ("w1", "w2")},
                          grads={"b1": torch.zeros(256, device="cuda")}),
        lambda: F.ce_fwd(x, head, t.int()), lambda: F.ce_fwd(x, head, t[:2]),
        lambda: F.ce_fwd(x, head[:, :32], t), lambda: F.ce_fwd(x, head.float(), t),
        lambda: F.ce_bwd(x, head, t, torch.zeros(4, device="cuda"), torch.zeros(3, device="cuda")),
        lambda: F.ce_bwd(x, head, t, torch.zeros(4, device="cuda"),
                         torch.ones(1, device="cuda").expand(4)),
        lambda: F.ce_bwd(x, head, t, torch.zeros(4, device="cuda"), torch.zeros(1)),
        lambda: F.ce_bwd(x, head, t, torch.zeros(4, device="cuda"), torch.zeros(1, device="cuda"),
                         dw=torch.zeros_like(head)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail("call %d was accepted" % i)
    # rules of the library itself: 16-byte pointers, multiples of 8, 8 bits with f32
    with pytest.raises(oz.OasesError) as e:
        flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
        F.glu_fwd(flat[1:].view(4, 64), w)
    assert e.value.status == 1
    with pytest.raises(oz.OasesError) as e:
        F.ce_fwd(torch.zeros(2, 12).bfloat16().cuda(), torch.zeros(5, 12).bfloat16().cuda(), t[:2])
    assert e.value.status == 2
    with pytest.raises(oz.OasesError) as e:
        wf = {k: v.float() for k, v in w.items()}
        F.glu_fwd(x.float(), wf, save="mxfp8")
    assert e.value.status == 2


@pytest.mark.parametrize("save", ["none", "pre", "mxfp8"])
def test_model_of_the_pieces_together(save):
    """Attention segment (DeviceBlock), gated feed-forward with LayerNorm and
    residual, head and loss: loss and every gradient against float64."""
    import ctypes

    import oracle
    from oracle.ops import layer_norm, layer_norm_backward
    from synth import BlockShape, block_inputs
    from tensor_model_transformer_tp_gb300.device import DeviceBlock, to_numpy

    shape = BlockShape("attn", "bf16", batch=2, seq=96, hidden=256, heads=2, w=2, sub_batches=2)
    M, H, Fn, V = shape.rows, shape.hidden, 520, 1009
    inp = block_inputs(shape, seed=4, affine=True)
    blk = DeviceBlock(shape, inp["layers"])
    x0 = blk.tensor(inp["x"])
    _, w, _, _ = glu_case("bf16", 1, H, Fn, True, False, seed=3)
    _, head, t, d = ce_case("bf16", M, H, V, True, seed=2)
    ln_g = (1 + 0.1 * torch.randn(H)).bfloat16().cuda()
    ln_b = (0.1 * torch.randn(H)).bfloat16().cuda()
    L = oz.lib()
    L.oases_debug_layer_norm.argtypes = [ctypes.c_void_p] * 6 + [ctypes.c_int] * 2 + [
        ctypes.c_float, ctypes.c_int, ctypes.c_void_p]
    L.oases_debug_layer_norm_bwd_scratch_bytes.restype = ctypes.c_size_t
    L.oases_debug_layer_norm_bwd.argtypes = [ctypes.c_void_p] * 9 + [ctypes.c_int] * 3 + [
        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]
    st = torch.cuda.current_stream().cuda_stream

    x1 = blk.fwd(x0)
    u = torch.empty_like(x1)
    mean, rstd = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    assert L.oases_debug_layer_norm(x1.data_ptr(), ln_g.data_ptr(), ln_b.data_ptr(), u.data_ptr(),
                                    mean.data_ptr(), rstd.data_ptr(), M, H, 1e-5, 1, st) == 0
    y, saved = F.glu_fwd(u, w, resid=x1, save=save)
    loss, lse = F.ce_fwd(y, head, t)
    dhead = torch.zeros(V, H, device="cuda")
    dy, _ = F.ce_bwd(y, head, t, lse, d, dw=dhead)
    gw = {k: torch.zeros_like(v, dtype=torch.float32) for k, v in w.items()}
    du, _ = F.glu_bwd(u, dy, w, save=save, saved=saved, grads=gw, dx_dtype=torch.float32)
    dx1, dg, db = torch.empty_like(x1), torch.zeros(H, device="cuda"), torch.zeros(H, device="cuda")
    nb = L.oases_debug_layer_norm_bwd_scratch_bytes(M, H)
    scratch = torch.empty(nb, dtype=torch.uint8, device="cuda")
    assert L.oases_debug_layer_norm_bwd(du.data_ptr(), x1.data_ptr(), mean.data_ptr(),
                                        rstd.data_ptr(), ln_g.data_ptr(), dy.data_ptr(),
                                        dx1.data_ptr(), dg.data_ptr(), db.data_ptr(), M, H, 1,
                                        scratch.data_ptr(), nb, st) == 0
    dx0 = blk.recompute_bwd(x0, dx1)
    torch.cuda.synchronize()
    oz.oases_check_device(None)

    # float64: the same chain; the attention segment through the oracle's step
    W, Hd, tt, D = {k: f64(v) for k, v in w.items()}, f64(head), t.cpu().numpy(), f64(d)
    X1 = oracle.run_step(shape, inp, mode="none")["y"]
    G, B = f64(ln_g), f64(ln_b)
    Un, mn, rs = layer_norm(X1, G, B, 1e-5)
    a, b = glu_projections(Un, W)
    Y = glu_output(a, b, W, "silu", X1)
    wl, _, _ = ce_forward(Y, Hd, tt)
    dY, dH, _ = ce_backward(Y, Hd, tt, D)
    if save == "mxfp8":
        a, b = kept_values(saved, save, M, Fn)
    dU, wg = glu_backward(dY, Un, a, b, W, "silu")
    dX1, dG, dB = layer_norm_backward(dU, X1, mn, rs, G)
    ref = oracle.run_step(shape, {**inp, "g": dX1 + dY}, mode="none")
    got = {"loss": loss, "dhead": dhead, "dx": dx0, "ln_g": dg, "ln_b": db,
           **{"f" + k: v for k, v in gw.items()}, **{"a" + k: v for k, v in blk.grads[0].items()}}
    want = {"loss": wl, "dhead": dH, "dx": ref["dx"], "ln_g": dG, "ln_b": dB,
            **{"f" + k: v for k, v in wg.items()}, **{"a" + k: v for k, v in ref["grads"][0].items()}}
    for k, v in want.items():
        # the block's own bf16 tolerance (rel-L2 2e-2) holds for the longer chain
        # too: a dozen bf16 roundings of 2^-9 rms each in series
        r = np.linalg.norm(to_numpy(got[k]) - v) / np.linalg.norm(v)
        assert r <= 2e-2, (k, r)
