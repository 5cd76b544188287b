"""Layer norm, the linear head's cross entropy and clipping at the ends of their ranges, against
plain 64-bit implementations.  Tolerances count roundings, as in test_gpu_training.py: U is half a
step of float32, HALF[t] half a step of type t."""
import math

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from unbiased_nvfp4_gradient_amd import training
from test_gpu_training import (BF16, DEV, F16, F32, HALF, TINY, U, ce_inputs, ce_reference,
                               check_ce, gen, randn, strided, within)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------- losses of confident tokens


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("t,v", [(1, 300), (40, 1000), (128, 300), (300, 1000), (600, 20000)])
def test_cross_entropy_of_confident_tokens(t, v, kind):
    """Logits 1024 + c of the target and 1024 of every other word, exact in FP32: the loss is
    log(1 + (v - 1) e^-c), and nothing of the logits' common size reaches its error."""
    print(f"case: confident tokens t={t} v={v} {kind}", flush=True)
    c = torch.arange(t, device=DEV, dtype=torch.float64) % 31 + 2
    h = torch.zeros((t, 64), device=DEV)
    h[:, 0], h[:, 1] = c.float(), 1.0
    w = torch.zeros((v, 64), device=DEV)
    w[:, 1] = 1024.0
    w[v // 2, 0] = 1.0
    target = torch.full((t,), v // 2, device=DEV)
    f = nv.linear_cross_entropy_forward(h.to(kind), w.to(kind), target, reduction="none")
    # sums of at most 64 + 1 + v / 128 terms and the joins' and the logarithm's own steps
    sums = U * (65 + v / 128 + 16)
    loss = torch.log1p((v - 1) * torch.exp(-c))
    within(f.loss, loss, sums + 8 * U * loss, "loss")
    lse = 1024.0 + c + loss
    within(f.lse, lse, 2 * U * lse + sums, "lse")


@pytest.mark.parametrize("t", [3, 100, 300])
def test_cross_entropy_of_the_largest_logits(t):
    # logits of 1.5 2^127 and 0: finite, and their products with log2 e are not.  The loss of the
    # first word is 0 and its gradient 0; of another the gradient is w of the first
    h = torch.full((t, 1), 1.5 * 2.0 ** 64, device=DEV, dtype=BF16)
    w = torch.zeros((300, 1), device=DEV, dtype=BF16)
    w[7] = 2.0 ** 63
    target = torch.full((t,), 7, device=DEV)
    target[1::3] = 11
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    assert bool((f.lse == 1.5 * 2.0 ** 127).all())
    assert torch.equal(f.loss, torch.where(target == 7, 0.0, 1.5 * 2.0 ** 127))
    b = nv.linear_cross_entropy_backward(torch.ones(1, device=DEV), h, w, target, f.lse,
                                         reduction="sum")
    assert torch.equal(b.dh[:, 0].float(), torch.where(target == 7, 0.0, 2.0 ** 63))
    n = int((target == 11).sum())
    want = torch.zeros(300, dtype=torch.float64, device=DEV)
    want[7], want[11] = n * 1.5 * 2.0 ** 64, -n * 1.5 * 2.0 ** 64
    within(b.dw[:, 0], want, HALF[BF16] * want.abs(), "dw")


# ------------------------------------------------------------------------------ large launches


def test_cross_entropy_more_tokens_than_a_launch_has_threads_for():
    # 2^26 + 7 tokens: 2^32 threads at 64 to a token
    t, v = (1 << 26) + 7, 3
    i = torch.arange(t, device=DEV)
    h = ((i % 61).float() / 16.0).to(BF16)[:, None]
    w = torch.tensor([[1.0], [-0.5], [0.25]], device=DEV, dtype=BF16)
    target = i % v
    target[i % 7 == 3] = -100
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    kinds = (torch.arange(61, device=DEV, dtype=torch.float64) / 16.0)[:, None] * w.double().T
    lse = torch.logsumexp(kinds, 1)               # logits are exact: 61 different tokens
    keep, k = target != -100, i % 61
    lse_off = U * (4 * lse + 65 + 16)
    within(f.lse, lse[k] * keep, lse_off[k], "lse")
    loss = (lse[:, None] - kinds)[k, target.clamp(min=0)] * keep
    within(f.loss, loss, 2 * lse_off[k], "loss")
    mean = nv.linear_cross_entropy_forward(h, w, target)
    want = float(loss.sum()) / int(keep.sum())
    assert abs(float(mean.loss) - want) <= float(2 * lse_off.max()) + U * want
    assert torch.equal(mean.lse, f.lse)


@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("t", [20, 130])
def test_cross_entropy_wider_rows_than_a_launch_has_groups_for(t, reduction):
    # 2^22 + 4097 columns: more than 65536 groups of 64; all but the first and last 8 are 0, whose
    # gradients are 0
    d, v = (1 << 22) + 4097, 5
    (h, w, target), g = ce_inputs(t, 16, v, BF16, 98, ignored=0.0)
    wide = [torch.zeros((len(x), d), device=DEV, dtype=BF16) for x in (h, w)]
    for x, y in zip((h, w), wide):
        y[:, :8], y[:, -8:] = x[:, :8], x[:, 8:]
    f = nv.linear_cross_entropy_forward(*wide, target, reduction=reduction)
    dloss = 0.5 + torch.rand(f.loss.shape, generator=g, device=DEV)
    b = nv.linear_cross_entropy_backward(dloss, *wide, target, f.lse, reduction=reduction)
    ref, off = ce_reference(h, w, target, dloss, -100, reduction)
    for name, got, want, tol in zip(("loss", "lse"), f, ref, off):
        within(got, want, tol, name)
    for name, got, want, tol in zip(("dh", "dw"), b, ref[2:], off[2:]):
        within(torch.cat((got[:, :8], got[:, -8:]), 1), want, tol, name)
        assert not got[:, 8:-8].any()


@pytest.mark.parametrize("bias_only", [False, True])
def test_layer_norm_longer_rows_than_a_launch_has_threads_for(bias_only):
    # sums of 2^27 + 37 columns: 2^32 threads at 32 to a column
    rows, n = 2, (1 << 27) + 37
    g = gen(97)
    x, dy = randn(g, rows, n).to(BF16), randn(g, rows, n).to(BF16)
    mean = torch.tensor([0.25, -0.5], device=DEV)
    rstd = torch.tensor([1.5, 0.75], device=DEV)
    w = None if bias_only else torch.full((n,), 0.5, device=DEV)
    r = nv.layer_norm_backward(dy, x, mean, rstd, w, bias=True, bias_type=F32)
    dyd = dy.double()
    within(r.dbias, dyd.sum(0), 2 * U * dyd.abs().sum(0), "dbias")
    if not bias_only:
        # (x - mean) rstd dy of two rows: three roundings of each and one of the sum
        terms = dyd * ((x.double() - mean.double()[:, None]) * rstd.double()[:, None])
        within(r.dweight, terms.sum(0), 5 * U * terms.abs().sum(0) + 1e-40, "dweight")


# -------------------------------------------------------------------------- heads in pieces


@pytest.mark.parametrize("t,d,v,second,pad,kind", [
    (130, 2560, 110000, 104704, 0, BF16),         # rows read as they lie
    (130, 2500, 111000, 105984, 1, BF16),         # rows copied: 2528 elements each
    (300, 4096, 140001, 65536, 8, F16)])          # two whole pieces and a part
def test_cross_entropy_forward_pieces(t, d, v, second, pad, kind):
    """A piece of the forward pass is 2^28 elements of the head's rows, in whole tiles of 256 words;
    `second` is where the second one begins.  Half of the targets lie past it, some next to it."""
    print(f"case: forward pieces t={t} d={d} v={v} pad={pad} {kind}", flush=True)
    assert second == (1 << 28) // (-(-d // 32) * 32) // 256 * 256 < v
    g = gen(92)
    target = torch.randint(v, (t,), generator=g, device=DEV)
    target[1::2] = second + torch.randint(v - second, (t // 2,), generator=g, device=DEV)
    target[:8] = torch.tensor([0, second - 1, second, second + 1, second + 255, second + 256, v - 2,
                               v - 1], device=DEV)
    target[9::10] = -100
    w = randn(g, v, d) * d ** -0.5
    # the largest logits of some tokens lie in the second piece and of others in the first
    h = randn(g, t, d) + 6.0 * torch.rand((t, 1), generator=g, device=DEV) * w[target.clamp(min=0)]
    h, w = strided(h.to(kind), pad), strided(w.to(kind), pad)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    keep = target != -100
    hd, wd = h.double(), w.double()
    logits = hd @ wd.T
    lse = torch.logsumexp(logits, 1)
    own = logits.gather(1, target.clamp(min=0)[:, None])[:, 0]
    logit_off = d * U * (hd.abs() @ wd.abs().T).max(1).values
    off = logit_off + U * (4 * lse.abs() + 4 * own.abs() + 16 + 65 + v / 128)
    within(f.lse, lse * keep, off, "lse")
    within(f.loss, (lse - own) * keep, 2 * off, "loss")


@pytest.mark.parametrize("t,d,v,pad", [(130, 2560, 110000, 0), (130, 2500, 111000, 1),
                                       (300, 4096, 140001, 8)])
def test_cross_entropy_forward_pieces_count_every_word_once(t, d, v, pad):
    # logits of four columns in eighths, exact in whatever order: the bound, 2e-4 at the most, is
    # below what 128 words of the 140001 add to lse (9e-4)
    g = gen(93)
    h, w = torch.zeros((t, d), device=DEV), torch.zeros((v, d), device=DEV)
    at = torch.tensor([0, d // 3, d // 2, d - 1], device=DEV)
    h[:, at] = torch.randint(-6, 7, (t, 4), generator=g, device=DEV).float() / 8
    w[:, at] = torch.randint(-6, 7, (v, 4), generator=g, device=DEV).float() / 8
    target = torch.randint(v, (t,), generator=g, device=DEV)
    logits = h[:, at].double() @ w[:, at].double().T
    h, w = strided(h.to(BF16), pad), strided(w.to(BF16), pad)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    lse = torch.logsumexp(logits, 1)
    own = logits.gather(1, target[:, None])[:, 0]
    off = U * (4 * lse + 4 * own.abs() + 16 + 65 + v / 128)
    within(f.lse, lse, off, "lse")
    within(f.loss, lse - own, 2 * off, "loss")


@pytest.mark.parametrize("t,d,v,reduction", [(4200, 96, 100000, "mean"), (4200, 72, 123001, "none")])
def test_cross_entropy_backward_pieces(t, d, v, reduction):
    # at 4200 tokens a piece of the backward pass is 61440 words: one and a part, two and a part
    assert (1 << 28) // (-(-t // 256) * 256) // 256 * 256 == 61440
    check_ce(t, d, v, BF16, reduction, ignored=0.1)


# ------------------------------------------------------------------- gradients of weighted tokens


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("t", [24, 50, 100, 300])
def test_cross_entropy_weight_of_a_token_is_not_rounded_into_dh(t, kind):
    """Targets that the model gives no probability: their q is -1, which 16 bits hold, so dh is
    off by its own rounding and the small probabilities', whatever the tokens' weights."""
    g = gen(90 + t)
    d, v, n = 64, 1000, 20
    w = randn(g, v, d)
    w[:n] = 16.0 * torch.sign(randn(g, n, d))
    w[:n, 0] = -16.0
    w = w.to(kind)
    h = 0.01 * randn(g, t, d)
    h[:, 0] = 0.5
    h = h.to(kind)
    target = torch.randint(n, (t,), generator=g, device=DEV)
    dloss = 1.0 + torch.rand((t,), generator=g, device=DEV)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction="none", need_dw=False)
    logits = h.double() @ w.double().T
    p = torch.softmax(logits, 1)
    own = p.gather(1, target[:, None])
    assert float(own.max()) < 2.0 ** -14          # half a step below 1 in float16 is 2^-12
    # p of FP32 logits and lse, rounded to 16 bits; the target's q is -1 and so off by p
    rel = 2 * (d * U * (h.double().abs() @ w.double().abs().T)
               + U * (65 + v / 128 + 16 + 8 * logits.abs().max()))
    q_off = p * (HALF[kind] + rel) + 2.0 ** -25 * 2.0 ** -15
    q_off.scatter_(1, target[:, None], own)
    q = p.scatter_add(1, target[:, None], torch.full_like(own, -1.0))
    share = dloss.double()[:, None]
    dh = share * (q @ w.double())
    off = share * (q_off @ w.double().abs() + (v + 64) * U * (q.abs() @ w.double().abs()))
    within(b.dh, dh, off + HALF[kind] * (1 + 2.0 ** -6) * (dh.abs() + off) + TINY[kind], "dh")


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("reduction", ["none", "mean"])
@pytest.mark.parametrize("t", [1, 2, 3, 13, 25, 33, 64, 65, 100, 128])
def test_cross_entropy_few_tokens_gradients_are_rounded_once(t, reduction, kind):
    """A few tokens' gradients can be single products, in which a rounding of q to 16 bits would be
    as large as the outputs' own: q there is held as the sum of two 16-bit numbers."""
    d, v = 72, 700
    (h, w, target), g = ce_inputs(t, d, v, kind, 60 + t, ignored=0.1 if t > 3 else 0.0, sharp=3.0)
    dloss = 0.2 + 1.8 * torch.rand((t if reduction == "none" else 1,), generator=g, device=DEV)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction=reduction)
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction=reduction)
    keep = target != -100
    hd, wd = torch.where(keep[:, None], h.double(), 0.0), w.double()
    logits = hd @ wd.T
    p = torch.softmax(logits, 1)
    y = target.clamp(min=0)[:, None]
    q = p.scatter_add(1, y, torch.full_like(p[:, :1], -1.0))
    n = max(int(keep.sum()), 1)
    share = (keep * dloss.double() / (n if reduction == "mean" else 1))[:, None]
    # p of FP32 logits and lse; two halves of q, the second one's rounding and float16's least step
    size = (hd.abs() @ wd.abs().T).max(1, keepdim=True).values
    rel = 4 * d * U * size + U * (65 + v / 128 + 32 + 12 * torch.logsumexp(logits, 1)[:, None].abs())
    q_off = p * rel + 2 * HALF[kind] ** 2 * q.abs() + 2 * U * q.abs()
    least = 2.0 ** -25 * 2.0 ** -15 if kind == F16 else 0.0
    off = HALF[kind] * (1 + 2.0 ** -6)
    dh, dw = share * (q @ wd), (share * q).T @ hd
    dh_off = share * ((q_off + least) @ wd.abs() + (v + 64) * U * (q.abs() @ wd.abs()))
    dw_off = (share * q_off + 2 * least * share.max()).T @ hd.abs() \
        + (t + 64) * U * ((share * q.abs()).T @ hd.abs())
    within(b.dh, dh, dh_off + off * (dh.abs() + dh_off) + TINY[kind], "dh")
    within(b.dw, dw, dw_off + off * (dw.abs() + dw_off) + TINY[kind], "dw")


@pytest.mark.parametrize("t", [3, 70, 200])
def test_cross_entropy_gradient_of_the_largest_weight(t):
    # a weight in the last binade of float32, whose gradients bfloat16 holds
    g = gen(91 + t)
    h, w = (2.0 ** -60 * randn(g, t, 64)).to(BF16), (2.0 ** -60 * randn(g, 300, 64)).to(BF16)
    target = torch.randint(300, (t,), generator=g, device=DEV)
    dloss = torch.rand((t,), generator=g, device=DEV)
    dloss[t // 2] = 1.5 * 2.0 ** 127
    f = nv.linear_cross_entropy_forward(h, w, target, reduction="none")
    b = nv.linear_cross_entropy_backward(dloss, h, w, target, f.lse, reduction="none")
    ref, off = ce_reference(h, w, target, dloss, -100, "none")
    within(b.dh, ref[2], off[2], "dh")
    within(b.dw, ref[3], off[3], "dw")


@pytest.mark.parametrize("reduction", ["none", "mean", "sum"])
@pytest.mark.parametrize("t", [5, 64, 128, 200])
def test_cross_entropy_no_token_counts_whatever_its_gradient(t, reduction):
    # a sum over no tokens is 0, and neither infinity nor NaN times it
    (h, w, target), _ = ce_inputs(t, 64, 300, BF16, 5, ignored=2.0)
    f = nv.linear_cross_entropy_forward(h, w, target, reduction=reduction)
    for bad in (math.inf, math.nan):
        b = nv.linear_cross_entropy_backward(torch.full_like(f.loss, bad), h, w, target, f.lse,
                                             reduction=reduction)
        assert not b.dh.any() and not b.dw.any()


# -------------------------------------------------------------------------------- clipped tensors


def test_clipping_is_seen_by_autograd():
    """Tensors that are written count a version: a backward pass that saved one is refused."""
    for out in (False, True):
        x = torch.full((64,), 3.0, device=DEV, requires_grad=True)
        y = 2.0 * x
        z = y.square().sum()                      # saves y
        held, other = y.detach(), torch.ones(64, device=DEV)
        before = other._version
        nv.grad_norm([held])
        assert held._version == y._version == 0
        if out:
            nv.clip_grads([other], 1.0, out=[held])
            assert other._version == before
        else:
            nv.clip_grads([held, other], 1.0)
            assert other._version == before + 1
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            z.backward()
    with torch.inference_mode():                  # tensors that count none
        t = torch.ones(64, device=DEV)
        nv.clip_grads([t], 1.0)
        assert abs(float(t[0]) - 0.125) < 1e-6


# ---------------------------------------------------------------------------------------- guards


class Guards:
    """Buffers between elements that no call may change."""

    def __init__(self):
        self.held = []

    def __call__(self, n, dtype):
        buf = torch.full((n + 2048,), 77.0, dtype=dtype, device=DEV)
        self.held.append((buf, n))
        return buf[1024:1024 + n]

    def intact(self):
        torch.cuda.synchronize()
        return all(bool((b[:1024] == 77.0).all()) and bool((b[1024 + n:] == 77.0).all())
                   for b, n in self.held)


@pytest.mark.parametrize("kind", [BF16, F16])
@pytest.mark.parametrize("t,d,v", [(1, 77, 389), (32, 65, 33), (33, 131, 1001), (64, 1, 1),
                                   (65, 517, 999), (128, 333, 4097), (129, 77, 389),
                                   (300, 259, 1283)])
def test_loss_stays_inside(t, d, v, kind):
    """Outputs and workspaces of both passes between guards: few tokens and tiles, odd sizes."""
    print(f"case: guarded loss t={t} d={d} v={v} {kind}", flush=True)
    L, st, code = training._lib(), torch.cuda.current_stream().cuda_stream, training.TYPES[kind]
    (h, w, target), g = ce_inputs(t, d, v, kind, 41)
    guard = Guards()
    loss, lse = guard(t, F32), guard(t, F32)
    dh, dw = guard(t * d, kind), guard(v * d, kind)
    dloss = 0.5 + torch.rand((t,), generator=g, device=DEV)
    args = (h.data_ptr(), d, w.data_ptr(), d, target.data_ptr())
    tail = (t, d, v, -100, 2)
    need = L.linear_cross_entropy_workspace_bytes(0, t, d, v)
    assert L.linear_cross_entropy_forward(code, *args, *tail, loss.data_ptr(), lse.data_ptr(),
                                          guard(need, torch.uint8).data_ptr(), need, st) == 0
    need = L.linear_cross_entropy_workspace_bytes(1, t, d, v)
    ws = guard(need, torch.uint8)
    for one, other in ((dh, dw), (dh, None), (None, dw)):
        assert L.linear_cross_entropy_backward(code, dloss.data_ptr(), *args, lse.data_ptr(), *tail,
                                               training._ptr(one), training._ptr(other),
                                               ws.data_ptr(), need, st) == 0
    assert guard.intact()
    ref, off = ce_reference(h, w, target, dloss, -100, "none")
    for name, got, want, tol in zip(("loss", "lse", "dh", "dw"),
                                    (loss, lse, dh.view(t, d), dw.view(v, d)), ref, off):
        within(got, want, tol, name)


@pytest.mark.parametrize("kind", [F32, BF16])
@pytest.mark.parametrize("rows,n", [(7, 1), (70, 13), (37, 251), (9, 509), (5, 1021), (3, 2049),
                                    (5, 4099), (3, 8193), (2, 16389), (2, 40003)])
def test_layer_norm_stays_inside(rows, n, kind):
    """Every layout of a row over threads, with rows that end inside an access."""
    print(f"case: guarded layer norm {rows}x{n} {kind}", flush=True)
    L, st, code = training._lib(), torch.cuda.current_stream().cuda_stream, training.TYPES[kind]
    g = gen(42)
    x, dy, w = randn(g, rows, n).to(kind), randn(g, rows, n).to(kind), randn(g, n)
    guard = Guards()
    y, dx, mean, rstd = guard(rows * n, kind), guard(rows * n, kind), guard(rows, F32), guard(rows, F32)
    dw, db = guard(n, F32), guard(n, F32)
    need = L.layer_norm_workspace_bytes(code, rows, n)
    ws = guard(need, torch.uint8)
    assert L.layer_norm_forward(code, 0, x.data_ptr(), w.data_ptr(), w.data_ptr(), rows, n, n, 1e-5,
                                y.data_ptr(), mean.data_ptr(), rstd.data_ptr(), st) == 0
    assert L.layer_norm_backward(code, 0, dy.data_ptr(), x.data_ptr(), mean.data_ptr(),
                                 rstd.data_ptr(), w.data_ptr(), rows, n, n, n, dx.data_ptr(),
                                 dw.data_ptr(), db.data_ptr(), ws.data_ptr(), need, st) == 0
    assert guard.intact()
    f = nv.layer_norm_forward(x, w, w)
    r = nv.layer_norm_backward(dy, x, f.mean, f.rstd, w, bias=True)
    for got, want in zip((y, mean, rstd, dx, dw, db), (*f, *r)):
        assert torch.equal(got, want.flatten())


@pytest.mark.parametrize("inf", [False, True])
@pytest.mark.parametrize("sizes", [[1, 5], [4099] * 9, [4095, 4096, 4097, 70001], [17] * 150 + [9001]])
def test_clipping_stays_inside(sizes, inf):
    """Outputs at odd places of one buffer, with elements between them that stay."""
    g = gen(43 + len(sizes))
    for kind in (F32, BF16, F16):
        grads = [randn(g, n).to(kind) for n in sizes]
        buf = torch.full((sum(sizes) + 3 * len(sizes) + 3,), 77.0, dtype=kind, device=DEV)
        mask = torch.ones_like(buf, dtype=torch.bool)
        out, at = [], 3
        for n in sizes:
            out.append(buf[at:at + n])
            mask[at:at + n] = False
            at += n + 3
        guard = Guards()
        norm_type = math.inf if inf else 2.0
        norm = nv.clip_grads(grads, 0.01, norm_type=norm_type, out=out)
        assert bool((buf[mask] == 77.0).all())
        inner = [guard(n, kind) for n in sizes[:9]]
        for t, x in zip(inner, grads):
            t.copy_(x)
        nv.clip_grads(inner, 0.01, norm_type=norm_type)
        assert guard.intact()
        for x, o in zip(grads, out):
            ref = x.double() * (0.01 / (float(norm) + 1e-6))
            tol = ref.abs() * (HALF[kind] * (1 + 2.0 ** -6) + 8 * U) + TINY[kind]
            within(o, ref, tol, "clipped")


@pytest.mark.parametrize("ignored", [0.0, 0.6, 2.0])
@pytest.mark.parametrize("t,d,v", [(5, 77, 389), (40, 128, 33), (100, 333, 4097), (200, 96, 700),
                                   (300, 64, 20000), (700, 520, 777)])
def test_loss_depends_on_nothing_left_in_its_workspace(t, d, v, ignored):
    # bytes that read as NaN in every type, and zeros
    L, st = training._lib(), torch.cuda.current_stream().cuda_stream
    (h, w, target), g = ce_inputs(t, d, v, BF16, 44, ignored=ignored)
    dloss = 0.5 + torch.rand((t,), generator=g, device=DEV)
    args, tail = (h.data_ptr(), d, w.data_ptr(), d, target.data_ptr()), (t, d, v, -100, 2)
    results = []
    for byte in (0, 255):
        out = [torch.empty(n, dtype=k, device=DEV) for n, k in ((t, F32), (t, F32), (t * d, BF16),
                                                               (v * d, BF16))]
        for back in (0, 1):
            need = L.linear_cross_entropy_workspace_bytes(back, t, d, v)
            ws = torch.full((need,), byte, dtype=torch.uint8, device=DEV)
            if back:
                rc = L.linear_cross_entropy_backward(1, dloss.data_ptr(), *args, out[1].data_ptr(),
                                                     *tail, out[2].data_ptr(), out[3].data_ptr(),
                                                     ws.data_ptr(), need, st)
            else:
                rc = L.linear_cross_entropy_forward(1, *args, *tail, out[0].data_ptr(),
                                                    out[1].data_ptr(), ws.data_ptr(), need, st)
            assert rc == 0
        results.append(out)
    assert all(torch.equal(a, b) and bool(a.isfinite().all()) for a, b in zip(*results))


def test_calls_on_a_stream_given_to_them():
    x = randn(gen(45), 40, 96).to(BF16)
    want = nv.layer_norm_forward(x)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = nv.layer_norm_forward(x, stream=side)
    norm = nv.grad_norm([x], stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.equal(norm, nv.grad_norm([x]))
