"""Layer norm, the linear head's cross entropy and gradient clipping on the GPU against plain
64-bit implementations.

Tolerances count roundings.  U = 2^-24 is half a step of float32, HALF[t] half a step of the
output's type.  A sum that a kernel forms by at most K additions in sequence is off by at most
K U times the sum of its terms' magnitudes.
"""
import importlib.util
import math
import os

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from unbiased_nvfp4_gradient_amd import training

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in HALF}   # least subnormal
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max())} " \
        f"above its bound (largest error {float(err.max())})"


def strided(t, pad, shift=0):
    """t as a view into a wider matrix whose other elements are NaN, starting at `shift`."""
    wide = torch.full((t.shape[0], t.shape[1] + pad + shift), float("nan"), dtype=t.dtype,
                      device=t.device)
    wide[:, shift:shift + t.shape[1]] = t
    return wide[:, shift:shift + t.shape[1]]


# ---------------------------------------------------------------------------------- layer norm

# serial additions of one thread, its wave and its workgroup: at most 32 + 6 + 16
K_ROW = 64


def check_layer_norm(rows, n, x_type, p_type, pad=0, weight=True, bias=True, shift=0.0, eps=1e-5,
                     seed=0):
    print(f"case: layer norm {rows}x{n} {x_type} {p_type} pad={pad} weight={weight} "
          f"bias={bias}", flush=True)
    g = gen(seed + 31 * rows + n)
    x = strided((randn(g, rows, n) * torch.exp(randn(g, n)) + shift).to(x_type), pad, pad % 2)
    dy = strided(randn(g, rows, n).to(x_type), pad)
    w = (1 + 0.3 * randn(g, n)).to(p_type) if weight else None
    b = (0.3 * randn(g, n)).to(p_type) if bias else None
    f = nv.layer_norm_forward(x, w, b, eps=eps)
    r = nv.layer_norm_backward(dy, x, f.mean, f.rstd, w, bias=bias)
    xd, dyd = x.double(), dy.double()
    wd = w.double() if weight else torch.ones(n, device=DEV, dtype=torch.float64)
    bd = b.double() if bias else torch.zeros(n, device=DEV, dtype=torch.float64)
    mean = xd.mean(1)
    var = (xd - mean[:, None]).square().mean(1)
    rstd = (var + eps).rsqrt()
    size = xd.abs().mean(1)
    within(f.mean, mean, (K_ROW + 2) * U * size, "mean")
    # a mean off by e moves the variance by e^2 only, beside the roundings of its own sum
    e = (K_ROW + 2) * U * size
    rel = (K_ROW + 8) * U + e ** 2 * rstd ** 2
    within(f.rstd, rstd, rel * rstd, "rstd")
    z = (xd - mean[:, None]) * rstd[:, None]
    y = z * wd + bd
    slack = (rel[:, None] + 8 * U) * (z * wd).abs() + (e * rstd)[:, None] * wd.abs() \
        + 4 * U * bd.abs()
    within(f.y, y, HALF[x_type] * (y.abs() + slack) + slack + TINY[x_type], "y")
    # the backward pass of the same saved statistics
    mean, rstd = f.mean.double()[:, None], f.rstd.double()[:, None]
    z = (xd - mean) * rstd
    gd = dyd * wd
    s1, s2 = gd.mean(1, keepdim=True), (gd * z).mean(1, keepdim=True)
    dx = rstd * (gd - s1 - z * s2)
    slack = (K_ROW + 8) * U * rstd * (gd.abs() + gd.abs().mean(1, keepdim=True)
                                      + z.abs() * (gd * z).abs().mean(1, keepdim=True))
    within(r.dx, dx, HALF[x_type] * (dx.abs() + slack) + slack + TINY[x_type], "dx")
    # a workgroup adds its rows (at most all / 512 + 1), its 4 waves, then 32 + 16 partial rows
    k = rows // 512 + 1 + 4 + 48 + 8
    if rows >= 512 and n > 16384:
        k = rows // 64 + 1 + 4 + 8
    if weight:
        ref, slack = (dyd * z).sum(0), k * U * (dyd * z).abs().sum(0)
        within(r.dweight, ref, HALF[p_type] * (ref.abs() + slack) + slack + TINY[p_type],
               "dweight")
    else:
        assert r.dweight is None
    if bias:
        ref, slack = dyd.sum(0), k * U * dyd.abs().sum(0)
        out = p_type if weight else x_type
        within(r.dbias, ref, HALF[out] * (ref.abs() + slack) + slack + TINY[out], "dbias")
    else:
        assert r.dbias is None


@pytest.mark.parametrize("x_type,p_type", [(F32, F32), (BF16, BF16), (BF16, F32), (F16, F16),
                                           (F16, F32)])
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (5, 512), (4, 513), (130, 1024), (9, 1025),
                                    (2, 2049), (700, 2048), (33, 4100), (17, 8192), (3, 16384)])
def test_layer_norm(rows, n, x_type, p_type):
    check_layer_norm(rows, n, x_type, p_type)


@pytest.mark.parametrize("x_type", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(5000, 16), (3001, 33), (2500, 64), (1000, 104), (999, 251),
                                    (2000, 256), (200000, 24), (1, 64), (66, 12)])
def test_layer_norm_of_several_rows_a_wave(rows, n, x_type):
    # more rows than one pass of the workgroups takes, rows that leave part of a wave without one
    check_layer_norm(rows, n, x_type, F32)


@pytest.mark.parametrize("x_type", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n,pad", [(7, 1023, 3), (5, 250, 1), (3, 4097, 5), (6, 64, 8)])
def test_layer_norm_strided(rows, n, pad, x_type):
    check_layer_norm(rows, n, x_type, x_type, pad=pad)


@pytest.mark.parametrize("weight,bias", [(False, False), (True, False), (False, True)])
def test_layer_norm_without_parameters(weight, bias):
    check_layer_norm(19, 300, BF16, BF16, weight=weight, bias=bias)


@pytest.mark.parametrize("rows,n,x_type", [(2, 40001, BF16), (600, 20000, F32), (1, 33000, F16)])
def test_layer_norm_long_rows(rows, n, x_type):
    check_layer_norm(rows, n, x_type, F32, pad=3)


def test_layer_norm_far_from_zero():
    # the variance is of differences from the mean, so a common offset does not cancel it away
    check_layer_norm(40, 1000, F32, F32, shift=1000.0)


def test_layer_norm_constant_rows_and_no_rows():
    x = torch.full((3, 100), 2.5, device=DEV, dtype=BF16)
    f = nv.layer_norm_forward(x, eps=1e-5)
    assert torch.equal(f.y, torch.zeros_like(x)) and torch.isfinite(f.rstd).all()
    e = torch.empty((0, 100), device=DEV, dtype=BF16)
    w = torch.ones(100, device=DEV, dtype=F32)
    f = nv.layer_norm_forward(e, w, w)
    r = nv.layer_norm_backward(e, e, f.mean, f.rstd, w, bias=True)
    assert f.y.shape == (0, 100) and r.dx.shape == (0, 100)
    assert not r.dweight.any() and not r.dbias.any()


def test_layer_norm_nan_stays_in_its_row():
    g = gen(3)
    x = randn(g, 6, 700).to(BF16)
    x[2, 5] = float("nan")
    y = nv.layer_norm_forward(x).y
    assert y[2].isnan().all() and not y[[0, 1, 3, 4, 5]].isnan().any()


def test_layer_norm_is_reproducible_and_shaped():
    g = gen(4)
    x, dy = randn(g, 4, 250, 384).to(BF16), randn(g, 4, 250, 384).to(BF16)
    w = randn(g, 384)
    a = nv.layer_norm_forward(x, w, w)
    r = nv.layer_norm_backward(dy, x, a.mean, a.rstd, w, bias=True)
    assert a.y.shape == x.shape and a.mean.shape == x.shape[:2]
    for _ in range(3):
        b = nv.layer_norm_forward(x, w, w)
        q = nv.layer_norm_backward(dy, x, b.mean, b.rstd, w, bias=True)
        assert all(torch.equal(u, v) for u, v in zip((*a, *r), (*b, *q)))


def test_layer_norm_autograd_against_differences():
    g = gen(5)
    x, dy = randn(g, 6, 40), randn(g, 6, 40)
    w, b = 1 + 0.2 * randn(g, 40), 0.2 * randn(g, 40)
    leaves = [t.requires_grad_() for t in (x, w, b)]
    nv.layer_norm(*leaves).backward(dy)

    def loss(*a):
        a = [t.double() for t in a]
        z = (a[0] - a[0].mean(1, keepdim=True)) * \
            (a[0].var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
        return float(((z * a[1] + a[2]) * dy.double()).sum())

    step = 1e-4                   # central differences in 64 bits: off by about step^2
    with torch.no_grad():
        for k, leaf in enumerate(leaves):
            d = randn(g, *leaf.shape)
            args = [[t.double() + (s * step * d.double() if i == k else 0)
                     for i, t in enumerate(leaves)] for s in (1, -1)]
            want = (loss(*args[0]) - loss(*args[1])) / (2 * step)
            got = float((leaf.grad.double() * d.double()).sum())
            assert abs(got - want) <= 1e-4 * float((leaf.grad * d).abs().sum()), (k, got, want)


def test_layer_norm_more_rows_than_a_launch_has_threads_for():
    # 2^26 + 5 rows of 4: 2^32 threads at a wave to a row
    rows = (1 << 26) + 5
    x = torch.zeros((rows, 4), device=DEV, dtype=BF16)
    x[:, 0] = 1.0
    f = nv.layer_norm_forward(x, eps=0.0)
    r = nv.layer_norm_backward(x, x, f.mean, f.rstd, bias=True)
    for i in (0, 1 << 25, rows - 1):
        assert torch.equal(f.y[i], f.y[1]) and float(f.mean[i]) == 0.25
        assert torch.equal(r.dx[i], r.dx[1])
    assert abs(float(f.y[rows - 1, 0]) - 3.0 ** 0.5) < 2.0 ** -7
    assert torch.equal(f.mean, f.mean[:1].expand(rows))


def test_layer_norm_autograd_of_some_parameters():
    g = gen(6)
    x, dy = randn(g, 300, 96).to(BF16), randn(g, 300, 96).to(BF16)
    w, b = randn(g, 96), randn(g, 96)
    # a bias alone, in float32: its gradient is not rounded to x's type on the way
    bias = b.clone().requires_grad_()
    nv.layer_norm(x, None, bias).backward(dy)
    ref = dy.double().sum(0)
    within(bias.grad, ref, 64 * U * dy.double().abs().sum(0), "dbias")
    # a weight that is not trained has no gradient, and the others are what they were
    leaf, bias = x.clone().requires_grad_(), b.clone().requires_grad_()
    nv.layer_norm(leaf, w, bias).backward(dy)
    f = nv.layer_norm_forward(x, w, b)
    r = nv.layer_norm_backward(dy, x, f.mean, f.rstd, w, bias=True)
    assert torch.equal(leaf.grad, r.dx) and torch.equal(bias.grad, r.dbias)
    assert nv.layer_norm_backward(dy, x, f.mean, f.rstd, w, need_dweight=False).dweight is None
    with pytest.raises(ValueError, match="bias_type"):
        nv.layer_norm_backward(dy, x, f.mean, f.rstd, w, bias=True, bias_type=BF16)
    # a second derivative is refused, not wrong
    dx, = torch.autograd.grad(nv.layer_norm(leaf, w, b).float().square().sum(), leaf,
                              create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


# ------------------------------------------------------------------------------- cross entropy


def ce_reference(h, w, target, dloss, ignore, reduction):
    """(loss, lse, dh, dw, bounds of loss, lse, dh, dw) in 64 bits."""
    kind = h.dtype
    hd, wd = h.double(), w.double()
    v, d = w.shape
    keep = (target != ignore)
    hd = torch.where(keep[:, None], hd, torch.zeros_like(hd))     # masked tokens reach nothing
    logits = hd @ wd.T
    # FP32 products and sums over d, in whatever order
    logit_off = d * U * (hd.abs() @ wd.abs().T).max(1).values
    lse = torch.logsumexp(logits, 1)
    y = target.clamp(0, v - 1)
    own = logits.gather(1, y[:, None])[:, 0]
    # exp2 and log2 of the hardware, the rounding of the scaled maximum, and sums of at most
    # 64 + 1 + v / 128 terms
    lse_off = logit_off + U * (4 * lse.abs() + 4 * own.abs() + 16 + 65 + v / 128)
    loss = (lse - own) * keep
    n = max(int(keep.sum()), 1)
    p = torch.exp(logits - lse[:, None])
    q = p.clone()
    q.scatter_add_(1, y[:, None], torch.full_like(q[:, :1], -1.0))
    share = keep.double() * (dloss.double() / (n if reduction == "mean" else 1))
    # p from the saved FP32 lse and FP32 logits, then q rounded to 16 bits
    rel = 2 * (logit_off + lse_off) + U * (16 + 4 * lse.abs())
    q_off = (HALF[kind] * q.abs() + (p * rel[:, None])) * share.abs()[:, None]
    if kind == F16:               # relative to the largest |share|, in units of 2^-15
        q_off = q_off + 2.0 ** -25 * 2.0 ** -15 * 2 * share.abs().max()
    q = q * share[:, None]
    dh, dw = q @ wd, q.T @ hd
    t = h.shape[0]
    dh_off = q_off @ wd.abs() + (v + 64) * U * (q.abs() @ wd.abs())
    dw_off = q_off.T @ hd.abs() + (t + 64) * U * (q.abs().T @ hd.abs())
    off = HALF[kind] * (1 + 2.0 ** -6)
    dh_off = dh_off + off * (dh.abs() + dh_off) + TINY[kind]
    dw_off = dw_off + off * (dw.abs() + dw_off) + TINY[kind]
    loss_off = (2 * lse_off) * keep
    if reduction != "none":
        k = n if reduction == "mean" else 1
        loss, loss_off = loss.sum()[None] / k, (loss_off.sum() / k + U * loss.sum().abs() / k)[None]
    return (loss, lse * keep, dh, dw), (loss_off, lse_off, dh_off, dw_off)


def ce_inputs(t, d, v, kind, seed, ignored=0.2, pad=0, sharp=4.0):
    g = gen(seed)
    w = randn(g, v, d) * d ** -0.5
    target = torch.randint(v, (t,), generator=g, device=DEV)
    h = randn(g, t, d) + sharp * torch.rand((t, 1), generator=g, device=DEV) * w[target]
    drop = torch.rand((t,), generator=g, device=DEV) < ignored
    target[drop] = -100
    h, w = h.to(kind), w.to(kind)
    h[drop] = float("nan")            # what stands in a token that does not count
    return (strided(h, pad), strided(w, pad), target), g


def check_ce(t, d, v, kind, reduction, seed=1, **kw):
    print(f"case: cross entropy t={t} d={d} v={v} {kind} {reduction} {kw}", flush=True)
    (h, w, target), g = ce_inputs(t, d, v, kind, seed, **kw)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction=reduction)
    dloss = 0.5 + torch.rand((t if reduction == "none" else 1,), generator=g, device=DEV)
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction=reduction)
    ref, off = ce_reference(h, w, target, dloss, -100, reduction)
    for name, got, want, tol in zip(("loss", "lse", "dh", "dw"), (*f, *b), ref, off):
        assert got.shape == want.shape
        within(got, want, tol, name)
    assert not b.dh[target == -100].any()
    return f, b


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
@pytest.mark.parametrize("t,d,v", [(1, 64, 256), (3, 8, 5), (7, 1, 1), (33, 72, 300),
                                   (256, 256, 512), (300, 200, 1000), (517, 520, 777)])
def test_cross_entropy(t, d, v, reduction, kind):
    check_ce(t, d, v, kind, reduction)


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("t,d,v,pad", [(65, 1001, 600, 1), (40, 128, 700, 8), (9, 63, 130, 3)])
def test_cross_entropy_strided(t, d, v, pad, kind):
    check_ce(t, d, v, kind, "none", pad=pad)


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("t", [1, 31, 32, 33, 64, 65, 128, 129])
def test_cross_entropy_around_few_tokens(t, kind):
    # blocks of 32 tokens that end full, one short and one over; words and columns that end
    # inside a step
    check_ce(t, 264, 391, kind, "mean", ignored=0.0)
    check_ce(t, 517, 1057, kind, "none", ignored=0.4, pad=t % 3)


@pytest.mark.parametrize("t,pad", [(33, 1), (64, 3), (100, 0), (128, 1)])
def test_cross_entropy_few_tokens_laid_out(t, pad):
    # a head of more than 2^24 elements: the tokens' rows are copied before the products
    check_ce(t, 424, 41003, BF16, "sum", pad=pad)


def test_cross_entropy_few_tokens_of_many_rows_past_32_bits():
    # the last words of the head lie past 2^31 elements and past 2^32 bytes
    v, d = 131072, 17000
    w = torch.zeros((v, d), device=DEV, dtype=BF16)
    w[v - 1, :8] = 1.0
    h = torch.zeros((2, d), device=DEV, dtype=BF16)
    h[:, :8] = 2.0
    target = torch.tensor([v - 1, 5], device=DEV)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    lse = math.log(math.exp(16.0) + v - 1)
    assert abs(float(f.loss[0]) - (lse - 16.0)) < 1e-5 and abs(float(f.loss[1]) - lse) < 1e-5
    b = nv.linear_cross_entropy_backward(torch.ones(2, device=DEV), h, w, target, f.lse,
                                         reduction="none")
    p = math.exp(16.0 - lse)
    want = 2.0 * ((p - 1.0) + p)             # of both tokens
    assert abs(float(b.dw[v - 1, 3]) - want) <= 2.0 ** -7 * (2.0 * (1 - p) + 2.0 * p)
    assert not b.dw[v - 1, 8:].any() and float(b.dw[5, 0]) < 0.0
    assert abs(float(b.dh[1, 0]) - p) <= 2.0 ** -6 * p and not b.dh[:, 8:].any()


@pytest.mark.parametrize("t,d,v", [(700, 2056, 8200), (2600, 4700, 700), (3000, 72, 5003)])
def test_cross_entropy_tile_sizes(t, d, v):
    # more than 192 tiles of 256 in dw, in dh and in the logits, fewer in the other products
    check_ce(t, d, v, BF16, "mean")


@pytest.mark.parametrize("t,d,v", [(300, 64, 1), (200, 96, 100), (700, 128, 129), (300, 32, 5003),
                                   (1000, 64, 30007)])
def test_cross_entropy_head_read_as_it_lies(t, d, v):
    # rows of whole steps of 32 at 16-byte boundaries: words that end inside and before a tile
    check_ce(t, d, v, BF16, "none", pad=8)
    check_ce(t, d, v, F16, "sum")


def test_cross_entropy_many_pieces():
    # 4200 tokens: a piece of the backward pass is some 30 thousand words
    check_ce(4200, 96, 62000, BF16, "mean")


def test_cross_entropy_long_head():
    # the forward pass takes this head in pieces too (131 thousand words of 1100 elements)
    (h, w, target), _ = ce_inputs(5, 1100, 130900, BF16, 3)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    ref, off = ce_reference(h, w, target, torch.ones(5, device=DEV), -100, "none")
    within(f.lse, ref[1], off[1], "lse")
    within(f.loss, ref[0], off[0], "loss")


@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
def test_cross_entropy_no_token_counts(reduction):
    (h, w, target), _ = ce_inputs(70, 64, 300, BF16, 5, ignored=2.0)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction=reduction)
    assert not f.loss.any() and not f.lse.any()
    dloss = torch.ones_like(f.loss)
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction=reduction)
    assert not b.dh.any() and not b.dw.any()
    (h, w, target) = (h[:0], w, target[:0])
    f = nv.linear_cross_entropy_forward(h, w, target, reduction=reduction)
    dloss = torch.ones_like(f.loss)
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction=reduction)
    assert not f.loss.any() and b.dh.shape == (0, 64) and not b.dw.any()


def test_cross_entropy_target_outside():
    (h, w, target), _ = ce_inputs(6, 64, 300, BF16, 6, ignored=0.0)
    target[1], target[4] = 300, -7
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    assert f.loss.isnan().tolist() == [False, True, False, False, True, False]
    assert f.lse.isfinite().all()
    b = nv.linear_cross_entropy_backward(torch.ones(6, device=DEV), h, w, target, f.lse,
                                         reduction="none")
    assert b.dh.isnan().all(1).tolist() == [False, True, False, False, True, False]
    assert b.dw.isnan().all()


def test_cross_entropy_large_and_infinite_logits():
    w = torch.zeros((300, 1), device=DEV, dtype=BF16)
    w[7] = 300.0
    h = torch.tensor([[200.0], [-200.0]], device=DEV, dtype=BF16)
    target = torch.tensor([7, 3], device=DEV)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    # one logit of 60000, and one of -60000 that is no part of the sum
    assert float(f.lse[0]) == 60000.0 and float(f.loss[0]) == 0.0
    assert abs(float(f.lse[1]) - math.log(299)) < 1e-5
    # a logit of plus infinity makes lse infinite, one of minus infinity is no part of it
    w[7] = float("inf")
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    assert float(f.lse[0]) == math.inf
    assert abs(float(f.lse[1]) - math.log(299)) < 1e-5
    # nothing but minus infinity
    f = nv.linear_cross_entropy_forward(h[1:], w[7:8].expand(300, 1).contiguous(), target[1:],
                                        reduction="none")
    assert float(f.lse[0]) == -math.inf


@pytest.mark.parametrize("t", [5, 300])
def test_cross_entropy_infinite_weight_stays_out_of_other_rows(t):
    # every logit of word 7 is minus infinity: no part of the softmax, no gradient of its row
    h = torch.ones((t, 64), device=DEV, dtype=BF16)
    w = randn(gen(2), 400, 64).to(BF16)
    w[7] = -math.inf
    target = torch.arange(t, device=DEV) % 5
    f = nv.linear_cross_entropy_forward(h, w, target)
    b = nv.linear_cross_entropy_backward(torch.ones(1, device=DEV), h, w, target, f.lse,
                                         need_dh=False)
    assert f.loss.isfinite().all() and not b.dw[7].any() and b.dw.isfinite().all()


def test_cross_entropy_one_loss_gradient_is_uneven():
    # gradients of the loss of very different sizes, zeros among them
    (h, w, target), g = ce_inputs(64, 64, 400, F16, 8)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    dloss = 10.0 ** (6 * torch.rand(64, generator=g, device=DEV) - 4)
    dloss[3] = 0.0
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction="none")
    ref, off = ce_reference(h, w, target, dloss, -100, "none")
    within(b.dh, ref[2], off[2], "dh")
    within(b.dw, ref[3], off[3], "dw")


def test_cross_entropy_autograd():
    (h, w, target), g = ce_inputs(90, 128, 500, BF16, 9)
    h, w = h.clone().requires_grad_(), w.clone().requires_grad_()
    loss = nv.linear_cross_entropy(h, w, target, reduction="none")
    (3.0 * loss.sum()).backward()                      # an expanded gradient
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    b = nv.linear_cross_entropy_backward(torch.full((90,), 3.0, device=DEV), h, w, target, f.lse,
                                         reduction="none")
    assert torch.equal(h.grad, b.dh) and torch.equal(w.grad, b.dw)
    only = nv.linear_cross_entropy(h.detach(), w, target)
    w.grad = None
    only.backward()
    f = nv.linear_cross_entropy_forward(h, w, target)
    b = nv.linear_cross_entropy_backward(torch.ones(1, device=DEV), h, w, target, f.lse,
                                         need_dh=False)
    assert b.dh is None and torch.equal(w.grad, b.dw)


def test_cross_entropy_is_reproducible_and_agrees_with_differences():
    f, b = check_ce(100, 64, 700, BF16, "sum", seed=11, ignored=0.0)
    for _ in range(3):
        f2, b2 = check_ce(100, 64, 700, BF16, "sum", seed=11, ignored=0.0)
        assert all(torch.equal(x, y) for x, y in zip((*f, *b), (*f2, *b2)))
    (h, w, target), g = ce_inputs(100, 64, 700, BF16, 11, ignored=0.0)
    dloss = 0.5 + torch.rand((1,), generator=g, device=DEV)

    def loss(hd, wd):
        z = hd @ wd.T
        return float((torch.logsumexp(z, 1) - z.gather(1, target[:, None])[:, 0]).sum()
                     * dloss[0].double())
    step = 1e-4
    for grad, which in ((b.dh, 0), (b.dw, 1)):
        dirn = randn(gen(12), *grad.shape).double()
        a = [[h.double() + (s * step * dirn if which == 0 else 0),
              w.double() + (s * step * dirn if which == 1 else 0)] for s in (1, -1)]
        want = (loss(*a[0]) - loss(*a[1])) / (2 * step)
        got = float((grad.double() * dirn).sum())
        # every element's rounding at the most, half a step of the output and of q
        assert abs(got - want) <= 3 * HALF[BF16] * float((grad.double() * dirn).abs().sum())


# ------------------------------------------------------------------------------------ clipping


def norm_reference(grads, inf):
    if inf:
        return max(float(t.double().abs().max()) for t in grads if t.numel())
    return math.sqrt(sum(float(t.double().square().sum()) for t in grads))


@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("types", [(F32,), (BF16,), (F16,), (F32, BF16, F16)])
@pytest.mark.parametrize("sizes", [[1], [9, 0, 5, 1025], [4099] * 9, [8192, 8193, 100003],
                                   [17] * 401 + [0] + [30001] * 5])
def test_norm_and_clip(sizes, types, inf):
    print(f"case: clip {len(sizes)} tensors {types} inf={inf}", flush=True)
    g = gen(len(sizes))
    grads = []
    for i, n in enumerate(sizes):       # slices at odd places of a larger buffer
        t = types[i % len(types)]
        grads.append((0.1 * randn(g, n + 3)).to(t)[i % 4:i % 4 + n])
    kind = math.inf if inf else 2.0
    want = norm_reference(grads, inf)
    got = nv.grad_norm(grads, norm_type=kind)
    assert got.shape == (1,) and abs(float(got) - want) <= 2 * U * want
    for max_norm in (0.5 * want, 2.0 * want, 0.0):
        out = [torch.full_like(t, 7.0) for t in grads]
        keep = [t.clone() for t in grads]
        n2 = nv.clip_grads(grads, max_norm, norm_type=kind, out=out)
        assert torch.equal(n2, got)
        c = min(1.0, max_norm / (want + 1e-6))
        for t, o, k in zip(grads, out, keep):
            assert torch.equal(t, k)
            ref = t.double() * c
            # the factor: the norm, its sum with 1e-6, the quotient, then the product
            tol = ref.abs() * (HALF[t.dtype] * (1 + 2.0 ** -6) + 8 * U) + TINY[t.dtype]
            within(o, ref, tol, "clipped")
            if max_norm > want:
                assert torch.equal(o, t)
        assert torch.equal(nv.clip_grads(keep, max_norm, norm_type=kind), got)
        assert all(torch.equal(a, b) for a, b in zip(keep, out))


def test_clip_refuses_lists_it_cannot_take():
    """Refusals of the binding, all before anything is launched."""
    a, b = torch.ones(64, device=DEV), torch.ones(64, device=DEV)
    for bad, what in (([a.view(8, 8).t()], "contiguous"), ([a.double()], "float32, bfloat16"),
                      ([a, b.cpu()], "on one GPU"), ([a, 3.0], "torch tensors"),
                      ([a.expand(4, 64)], "contiguous"), ([a.to_sparse()], "contiguous")):
        with pytest.raises(ValueError, match=what):
            nv.grad_norm(bad)
        with pytest.raises(ValueError, match=what):
            nv.clip_grads(bad, 1.0)
    for out, what in (([a], "must hold 2"), ([a, b[:5]], "must match"),
                      ([a, b.to(BF16)], "must match")):
        with pytest.raises(ValueError, match=what):
            nv.clip_grads([torch.ones(64, device=DEV), torch.ones(64, device=DEV)], 1.0, out=out)
    for grads, out in (([a, a], None), ([a[:40], a[39:]], None), ([a, b], [b, a]),
                       ([a[:63], b[:63]], [a[1:], b[1:]])):
        with pytest.raises(nv.NVFP4Error):
            nv.clip_grads(grads, 1.0, out=out)
    assert torch.equal(a, torch.ones_like(a)) and torch.equal(b, torch.ones_like(b))
    # parameters of a module, which are tensors of another class, and slices side by side
    p = torch.nn.Parameter(torch.ones(16, device=DEV))
    assert abs(float(nv.grad_norm([p])) - 4.0) < 1e-6
    assert float(nv.clip_grads([a[:32], a[32:]], 100.0)) == 8.0


def test_norm_of_extreme_values():
    big = torch.full((5000,), 3e30, device=DEV)
    small = torch.full((5000,), 2e-30, device=DEV)
    assert abs(float(nv.grad_norm([big])) / (3e30 * math.sqrt(5000)) - 1) < 1e-6
    assert abs(float(nv.grad_norm([small])) / (2e-30 * math.sqrt(5000)) - 1) < 1e-6
    for bad in (float("nan"), float("inf")):
        t = torch.ones(9000, device=DEV)
        t[8765] = bad
        for kind in (2.0, math.inf):
            n = float(nv.grad_norm([small, t], norm_type=kind))
            assert math.isnan(n) if math.isnan(bad) else n == math.inf
    t = torch.ones(9, device=DEV)
    t[2] = float("nan")
    other = torch.ones(9, device=DEV)
    nv.clip_grads([t, other], 1.0)
    assert other.isnan().all()


def test_norm_past_32_bits():
    # an offset past 2^31 elements, the only element that is not 0 at the end
    n = (1 << 31) + 4097
    t = torch.zeros(n, device=DEV, dtype=BF16)
    t[-1] = 3.0
    t[5] = 4.0
    assert float(nv.grad_norm([t])) == 5.0
    nv.clip_grads([t], 2.5)
    assert float(t[-1]) == 1.5 and float(t[5]) == 2.0 and float(t[-2]) == 0.0


# ------------------------------------------------------------------------------------ together


def test_other_stream_and_graph():
    """The whole sequence on a side stream and captured into a graph; replays, with eager work
    between them, give the eager results."""
    g = gen(21)
    t, d, v = 200, 256, 1100
    x = randn(g, t, d).to(BF16)
    ln_w = 1 + 0.1 * randn(g, d)
    head = (randn(g, v, d) * d ** -0.5).to(BF16)
    target = torch.randint(v, (t,), generator=g, device=DEV)
    target[::9] = -100
    dloss = torch.ones(1, device=DEV)

    def step():
        f = nv.layer_norm_forward(x, ln_w)
        c = nv.linear_cross_entropy_forward(f.y, head, target)
        b = nv.linear_cross_entropy_backward(dloss, f.y, head, target, c.lse)
        r = nv.layer_norm_backward(b.dh, x, f.mean, f.rstd, ln_w)
        norm = nv.clip_grads([b.dw, r.dweight, r.dx], 0.01)
        return [f.y, c.loss, c.lse, b.dh, b.dw, r.dx, r.dweight, norm]

    eager = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(eager, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        x.copy_(randn(gen(30 + k), t, d).to(BF16))
        eager = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, held)), k


def test_backward_pass_captured():
    """Loss and backward pass through autograd in a graph; replays give the eager gradients."""
    g = gen(50)
    t, d, v = 140, 128, 700
    x = randn(g, t, d).to(BF16)
    target = torch.randint(v, (t,), generator=g, device=DEV)
    leaves = [(1 + 0.1 * randn(g, d)).requires_grad_(), (0.1 * randn(g, d)).requires_grad_(),
              (randn(g, v, d) * d ** -0.5).to(BF16).requires_grad_()]

    def step():
        loss = nv.linear_cross_entropy(nv.layer_norm(x, *leaves[:2]), leaves[2], target)
        loss.backward()
        return loss.detach()

    def eager():
        for leaf in leaves:
            leaf.grad = None
        return [step(), *(leaf.grad for leaf in leaves)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        eager()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for leaf in leaves:
        leaf.grad = None
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step()
    held = [loss, *(leaf.grad for leaf in leaves)]
    for k in range(4):
        x.copy_(randn(gen(60 + k), t, d).to(BF16))
        want = [u.clone() for u in eager()]
        torch.cuda.synchronize()
        for u in held[1:]:
            u.fill_(7.0)            # captured where there was no gradient: replaced, not added to
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), k


def test_example_learns():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    spec = importlib.util.spec_from_file_location(
        "train_step_example", os.path.join(root, "examples", "train_step.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    losses, norms = example.train(60)
    print(f"losses {losses[0]:.3f} {losses[-1]:.3f}", flush=True)
    assert all(map(math.isfinite, losses + norms)) and min(norms) > 0.0
    # one answer in ten is noise: it starts at a uniform guess or above and ends well below
    assert losses[0] > math.log(500) - 0.5 and losses[-1] < 0.7 * math.log(500)


@pytest.mark.parametrize("t", [20, 100])
def test_few_tokens_captured(t):
    """The kernels for few tokens in a graph: the tokens that count change between replays."""
    (h, w, target), g = ce_inputs(t, 192, 1003, BF16, 70)
    dloss = torch.ones(1, device=DEV)

    def step():
        f = nv.linear_cross_entropy_forward(h, w, target)
        b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse)
        return [*f, *b]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for k in range(4):
        h.copy_(randn(gen(80 + k), t, 192).to(BF16))
        target.copy_(torch.randint(1003, (t,), generator=g, device=DEV))
        target[k::k + 2] = -100
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, held)), k


def test_cross_entropy_tiles_agree_with_differences():
    (h, w, target), g = ce_inputs(300, 96, 600, BF16, 12, ignored=0.0)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="sum")
    b = nv.linear_cross_entropy_backward(torch.ones(1, device=DEV), h, w, target, f.lse,
                                         reduction="sum")

    def loss(hd, wd):
        z = hd @ wd.T
        return float((torch.logsumexp(z, 1) - z.gather(1, target[:, None])[:, 0]).sum())
    step = 1e-4
    for grad, which in ((b.dh, 0), (b.dw, 1)):
        dirn = randn(gen(13), *grad.shape).double()
        a = [[h.double() + (s * step * dirn if which == 0 else 0),
              w.double() + (s * step * dirn if which == 1 else 0)] for s in (1, -1)]
        want = (loss(*a[0]) - loss(*a[1])) / (2 * step)
        got = float((grad.double() * dirn).sum())
        # every element's rounding at the most, half a step of the output and of q
        assert abs(got - want) <= 3 * HALF[BF16] * float((grad.double() * dirn).abs().sum())


def test_outputs_stay_inside():
    """Outputs of odd sizes between guard elements, through the C ABI."""
    L = training._lib()
    st = torch.cuda.current_stream().cuda_stream
    g = gen(40)

    def guarded(n, dtype):
        buf = torch.full((n + 2048,), 77.0, dtype=dtype, device=DEV)
        return buf, buf[1024:1024 + n]

    def intact(buf, n):
        return bool((buf[:1024] == 77.0).all()) and bool((buf[1024 + n:] == 77.0).all())

    rows, n = 5, 1027
    x, dy = randn(g, rows, n).to(F16), randn(g, rows, n).to(F16)
    w = randn(g, n)
    bufs = [(guarded(rows * n, F16), rows * n), (guarded(rows, F32), rows),
            (guarded(rows, F32), rows), (guarded(rows * n, F16), rows * n),
            (guarded(n, F32), n), (guarded(n, F32), n)]
    y, mean, rstd, dx, dw, db = (b[0][1] for b in bufs)
    need = L.layer_norm_workspace_bytes(2, rows, n)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    assert L.layer_norm_forward(2, 0, x.data_ptr(), w.data_ptr(), w.data_ptr(), rows, n, n, 1e-5,
                                y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), st) == 0
    assert L.layer_norm_backward(2, 0, dy.data_ptr(), x.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), w.data_ptr(), rows, n, n, n, dx.data_ptr(),
                                 dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need, st) == 0
    t, d, v = 131, 77, 389
    (h, head, target), _ = ce_inputs(t, d, v, BF16, 41)
    ce = [(guarded(t, F32), t), (guarded(t, F32), t), (guarded(t * d, BF16), t * d),
          (guarded(v * d, BF16), v * d)]
    loss, lse, dh, dhead = (b[0][1] for b in ce)
    for back in (0, 1):
        need = L.linear_cross_entropy_workspace_bytes(back, t, d, v)
        ws, inner = guarded(need, torch.uint8)
        args = (h.data_ptr(), d, head.data_ptr(), d, target.data_ptr())
        tail = (t, d, v, -100, 2)
        if back:
            rc = L.linear_cross_entropy_backward(1, loss.data_ptr(), *args, lse.data_ptr(), *tail,
                                                 dh.data_ptr(), dhead.data_ptr(),
                                                 inner.data_ptr(), need, st)
        else:
            rc = L.linear_cross_entropy_forward(1, *args, *tail, loss.data_ptr(), lse.data_ptr(),
                                                inner.data_ptr(), need, st)
        assert rc == 0
        torch.cuda.synchronize()
        assert intact(ws, need)
    assert all(intact(b[0][0], b[1]) for b in (*bufs, *ce))
