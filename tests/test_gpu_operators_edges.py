"""Edges of the gated feed-forward block (oases_glu.h) and the linear head's cross
entropy (oases_ce.h) on the GPU: values and sizes at the ends of what the headers
allow."""
import itertools

import numpy as np
import pytest
import torch

import tensor_model_transformer_tp_gb300 as oz
from tensor_model_transformer_tp_gb300 import functional as F

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    oz.build_library()


def ce_tensors(dtype, M, H, V, seed=0):
    gen = torch.Generator().manual_seed(seed + M + 3 * H + 5 * V)
    x = torch.randn(M, H, generator=gen).to(T[dtype]).cuda()
    w = (torch.randn(V, H, generator=gen) * H ** -0.5).to(T[dtype]).cuda()
    t = torch.randint(0, V, (M,), generator=gen)
    t[::3] = -100
    return x, w, t.cuda()


# ---- one dloss for all rows that is infinite or NaN ------------------------------
# (37 x 40000: dx in split parts; 8000 x 20001: several pieces of the vocabulary)
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("dtype,M,H,V", [("bf16", 12, 64, 300), ("bf16", 140, 72, 901),
                                         ("bf16", 37, 64, 40000), ("bf16", 8000, 64, 20001),
                                         ("f32", 12, 33, 301), ("f32", 140, 64, 900)])
def test_ce_non_finite_dloss_of_all_rows_stays_in_the_rows_with_a_loss(dtype, M, H, V, value):
    x, w, t = ce_tensors(dtype, M, H, V)
    d = torch.full((1,), value, device="cuda")
    _, lse = F.ce_fwd(x, w, t)
    dx, dw = F.ce_bwd(x, w, t, lse, d)
    ignored = t == -100
    assert not dx[ignored].any()                         # 0, not NaN
    assert not torch.isfinite(dx[~ignored]).any() and not torch.isfinite(dw).any()
    # every row ignored (the mean over no rows: 1 / 0): no gradient at all
    none = torch.full_like(t, -100)
    start = torch.randn_like(w, dtype=torch.float32)
    acc = start.clone()
    dx, dw = F.ce_bwd(x, w, none, lse, d)
    assert not dx.any() and not dw.any()
    dx, _ = F.ce_bwd(x, w, none, lse, d, dw=acc)
    assert not dx.any() and torch.equal(acc, start)


# ---- few rows and more weight rows than a grid's second dimension has tiles ------
def block_64(x, w, dy):
    """(y, dx, dw1, dw2) of the block (SiLU, no biases) in float64."""
    x, w1, w2, dy = x.double(), w["w1"].double(), w["w2"].double(), dy.double()
    Fn = w2.shape[1]
    p = x @ w1.t()
    a, b = p[:, :Fn], p[:, Fn:]
    s = torch.sigmoid(a)
    h, dh = a * s * b, dy @ w2
    dp = torch.cat([dh * b * s * (1 + a * (1 - s)), dh * a * s], dim=1)
    return h @ w2.t(), dp @ w1, dp.t() @ x, dy.t() @ h


@pytest.mark.parametrize("save", ["none", "pre", "mxfp8"])
@pytest.mark.parametrize("H,Fn", [(8, 65536 * 64 - 56), (65535 * 128 + 8, 8)])
def test_glu_few_rows_of_very_wide_weights(H, Fn, save):
    """65536 tiles of 64 columns of ffn, and 65536 of 128 of hidden; as with 129
    rows, to two bf16 roundings (h, and y itself) of 2^-9 rms each.  The gradients
    rest on a, b and dh, sums over hidden in one chain of hidden / 16 matrix
    instructions: each drops what is below the accumulator's last bit, up to 2^-23 of
    a partial sum, and the partial sums of independent terms are in the mean square
    no larger than the whole one.  So the three factors are off by hidden / 16 2^-23
    each at most (1/16 at hidden 8388488, nothing at hidden 8)."""
    gen = torch.Generator(device="cuda").manual_seed(H)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

    x, dy = rnd(2, H), rnd(2, H)
    w = {"w1": rnd(2 * Fn, H, std=H ** -0.5), "w2": rnd(H, Fn, std=Fn ** -0.5)}
    y, saved = F.glu_fwd(x, w, save=save)
    oz.oases_check_device(torch.cuda.current_stream())
    want, wdx, wdw1, wdw2 = block_64(x, w, dy)
    assert float((y.double() - want).norm() / want.norm()) <= 2.0 ** -8
    if save != "none":
        return      # the kept values and the backward pass at them: the same kernels at any size
    dx, grads = F.glu_bwd(x, dy, w, save=save, saved=saved)
    for got, ref in ((dx, wdx), (grads["w1"], wdw1), (grads["w2"], wdw2)):
        assert float((got.double() - ref).norm() / ref.norm()) <= 2.0 ** -8 + 3 * H / 16 * 2.0 ** -23


# ---- a gradient does not depend on which others are wanted ------------------------
@pytest.mark.parametrize("dtype,M,H,Fn", [("f32", 256, 256, 1024), ("f32", 100, 520, 2048),
                                          ("f32", 2000, 64, 96), ("bf16", 256, 256, 1024),
                                          ("bf16", 3000, 136, 264)])
def test_glu_gradients_are_the_same_bits_whichever_are_wanted(dtype, M, H, Fn):
    gen = torch.Generator().manual_seed(M + H)

    def rnd(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen) * std).to(T[dtype]).cuda()

    x, dy = rnd(M, H), rnd(M, H)
    w = {"w1": rnd(2 * Fn, H, std=H ** -0.5), "w2": rnd(H, Fn, std=Fn ** -0.5), "b1": rnd(2 * Fn),
         "b2": rnd(H)}
    _, saved = F.glu_fwd(x, w, save="pre")

    def run(names, need_dx):
        grads = {k: torch.zeros_like(w[k], dtype=torch.float32) for k in names}
        dx, _ = F.glu_bwd(x, dy, w, save="pre", saved=saved, grads=grads, need_dx=need_dx)
        return dx, grads

    dx0, all_ = run(sorted(w), True)
    for n in range(len(w) + 1):
        for names in itertools.combinations(sorted(w), n):
            for need_dx in (False, True):
                dx, grads = run(names, need_dx)
                assert dx is None or torch.equal(dx, dx0), (names, need_dx)
                for k in names:
                    assert torch.equal(grads[k], all_[k]), (k, names, need_dx)


@pytest.mark.parametrize("dtype,M,H,V", [("f32", 250, 256, 1003), ("f32", 512, 512, 3000),
                                         ("f32", 60, 1024, 5000), ("bf16", 250, 256, 1003),
                                         ("bf16", 2500, 72, 3000)])
def test_ce_gradients_are_the_same_bits_whichever_are_wanted(dtype, M, H, V):
    x, w, t = ce_tensors(dtype, M, H, V)
    d = torch.full((1,), 1.0 / M, device="cuda")
    _, lse = F.ce_fwd(x, w, t)
    dx0, dw0 = F.ce_bwd(x, w, t, lse, d)
    assert torch.equal(F.ce_bwd(x, w, t, lse, d, need_dw=False)[0], dx0)
    assert torch.equal(F.ce_bwd(x, w, t, lse, d, need_dx=False)[1], dw0)


# ---- rows whose probability is all at one column ----------------------------------
CE_ONE = [("bf16", 5, 64), ("bf16", 300, 72), ("f32", 5, 33), ("f32", 130, 64)]


@pytest.mark.parametrize("dtype,M,H", CE_ONE)
def test_ce_vocabulary_of_one(dtype, M, H):
    """The softmax of one logit is 1: no loss, and lse is the logit (sums of
    products of whole numbers, exact in fp32)."""
    gen = torch.Generator().manual_seed(M)
    x = torch.randint(-3, 4, (M, H), generator=gen).to(T[dtype]).cuda()
    w = torch.randint(-60, 61, (1, H), generator=gen).to(T[dtype]).cuda()
    t = torch.zeros(M, dtype=torch.int64, device="cuda")
    loss, lse = F.ce_fwd(x, w, t)
    assert not loss.any()
    assert torch.equal(lse.double(), (x.double() @ w.double().t())[:, 0])


@pytest.mark.parametrize("V", [2, 300, 1009])
@pytest.mark.parametrize("dtype,M,H", CE_ONE)
def test_ce_one_logit_far_above_the_others(dtype, M, H, V):
    """Logits are whole numbers below 2^24; the target's is above the others by
    1000 and more, so the others' share is below e^-1000."""
    gen = torch.Generator().manual_seed(M + V)
    x = torch.randint(1, 4, (M, H), generator=gen).to(T[dtype]).cuda()
    w = torch.randint(-1, 2, (V, H), generator=gen)
    hot = V // 2
    w[hot] = torch.randint(50, 121, (H,), generator=gen)
    w = w.to(T[dtype]).cuda()
    t = torch.full((M,), hot, dtype=torch.int64, device="cuda")
    loss, lse = F.ce_fwd(x, w, t)
    l = x.double() @ w.double().t()
    assert float((l[:, hot:hot + 1] - l[:, [v for v in range(V) if v != hot]]).min()) > 1000
    assert not loss.any() and torch.equal(lse.double(), l[:, hot])


@pytest.mark.parametrize("dtype,M,H", CE_ONE)
def test_ce_loss_is_never_negative(dtype, M, H):
    """Large logits, the target's among the largest: lse is no less than any of them."""
    gen = torch.Generator().manual_seed(H)
    x = (torch.randn(M, H, generator=gen) * 100).to(T[dtype]).cuda()
    w = torch.randn(517, H, generator=gen).to(T[dtype]).cuda()
    t = (x.float() @ w.float().t()).argmax(dim=1)
    loss, lse = F.ce_fwd(x, w, t)
    assert (loss >= 0).all()
    # loss and lse are fp32 sums of the same logits: lse = logit + loss
    assert torch.isfinite(lse).all()


@pytest.mark.parametrize("V", [1, 2, 300, 1009])
@pytest.mark.parametrize("dtype,M,H", CE_ONE)
def test_ce_no_gradient_where_the_probability_is_one(dtype, M, H, V):
    """As above; the softmax is exactly the target's indicator, so g is 0."""
    gen = torch.Generator().manual_seed(M + V)
    x = torch.randint(1, 4, (M, H), generator=gen).to(T[dtype]).cuda()
    w = torch.randint(-1, 2, (V, H), generator=gen)
    w[V // 2] = torch.randint(50, 121, (H,), generator=gen)
    w = w.to(T[dtype]).cuda()
    t = torch.full((M,), V // 2, dtype=torch.int64, device="cuda")
    lse = (x.double() @ w.double().t())[:, V // 2].float()
    for d in (torch.ones(1, device="cuda"), torch.rand(M, generator=gen).cuda()):
        dx, dw = F.ce_bwd(x, w, t, lse, d)
        assert not dx.any() and not dw.any()


# ---- fp32 GeLU ---------------------------------------------------------------------
def test_glu_fp32_gelu_keeps_its_relative_accuracy_in_the_tail():
    """Wg = I, Wu = 0, bu = 1, W2 = I: y = gelu(x) and dx = dy gelu'(x), one fp32
    value each.  With z = a / sqrt(2): the complementary error function is good to 4
    ulp, z to 1.25 2^-24 relative, which counts 2 z^2 + 1 <= 26 times for |a| <= 5; the
    exponential to 2 ulp, a^2 / 2 <= 12.5 to 2^-24 relative; a handful of products:
    32 2^-23 covers each of Phi and phi."""
    n = 512
    a = torch.linspace(-5, 5, n).cuda().repeat(3, 1).contiguous()
    a[1:] += torch.tensor([[0.003], [0.007]], device="cuda")
    eye = torch.eye(n, device="cuda")
    w = {"w1": torch.cat([eye, torch.zeros_like(eye)]),
         "b1": torch.cat([torch.zeros(n), torch.ones(n)]).cuda(), "w2": eye}
    dy = torch.full_like(a, 1.0)
    A = a.double()
    cdf = 0.5 * torch.special.erfc(-A * 0.5 ** 0.5)
    pdf = torch.exp(-0.5 * A * A) * (2 * np.pi) ** -0.5
    for save in ("pre", "none"):
        y, saved = F.glu_fwd(a, w, act="gelu", save=save)
        dx, _ = F.glu_bwd(a, dy, w, act="gelu", save=save, saved=saved)
        assert ((y.double() - A * cdf).abs() <= 32 * 2.0 ** -23 * (A * cdf).abs()).all()
        assert ((dx.double() - (cdf + A * pdf)).abs()
                <= 32 * 2.0 ** -23 * (cdf + (A * pdf).abs())).all()
