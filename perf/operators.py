"""Cases for timing the operators around the quantized linear layer in a training step: layer
norm (forward and backward), softmax cross entropy of a linear head over a large vocabulary
(forward, and forward with gradients) and the global gradient norm with clipping.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where `own` is true, with this package's kernels; `exact` gives the same
results from the definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
IGNORE = -100


def listed():
    return [
        # the last norm of a few sequences that each produce one token: latency
        dict(name="ln fwd 5x2048 bf16", op="ln", dir="fwd", rows=5, n=2048, x="bf16", p="bf16",
             pad=0),
        # odd rows of an odd width, views of a wider tensor (rows not 16-byte aligned)
        dict(name="ln bwd 4099x1023 f16", op="ln", dir="bwd", rows=4099, n=1023, x="f16",
             p="f16", pad=3),
        # a norm of the 1.9B model's training step (32768 tokens, hidden 2048), float32 weights
        dict(name="ln train 32768x2048 bf16", op="ln", dir="train", rows=32768, n=2048,
             x="bf16", p="f32", pad=0),
        # the repository's largest activation in float32
        dict(name="ln bwd 16384x8192 f32", op="ln", dir="bwd", rows=16384, n=8192, x="f32",
             p="f32", pad=0),
        # the loss of a handful of held-out tokens: reads the head once
        dict(name="ce fwd 7x1024x8192 bf16", op="ce", dir="fwd", t=7, d=1024, v=8192, x="bf16",
             red="none", pad=0),
        # a short training batch
        dict(name="ce train 2048x2048x32768 bf16", op="ce", dir="train", t=2048, d=2048,
             v=32768, x="bf16", red="mean", pad=0),
        # odd everything, a weight per token, float16 under loss scaling
        dict(name="ce train 1537x1000x50001 f16", op="ce", dir="train", t=1537, d=1000, v=50001,
             x="f16", red="none", pad=8),
        # a long training batch over a large vocabulary
        dict(name="ce train 8192x2048x131072 bf16", op="ce", dir="train", t=8192, d=2048,
             v=131072, x="bf16", red="mean", pad=0),
        # the gradients of one small layer: latency
        dict(name="norm 9x4099 f32", op="grad", dir="norm", count=9, size=4099, spread=1.0,
             x="f32", inf=False),
        # every matrix of the 1.9B model's 24 layers (168 of them)
        dict(name="norm 168x8388608 bf16", op="grad", dir="norm", count=168, size=8388608,
             spread=1.0, x="bf16", inf=False),
        # many tensors of very different sizes, unaligned slices of one flat buffer
        dict(name="clip 300x40001 f32", op="grad", dir="clip", count=300, size=40001,
             spread=100.0, x="f32", inf=False),
        # large matrices clipped into a flat buffer of bfloat16
        dict(name="clip 24x16777216 bf16", op="grad", dir="clip", count=24, size=16777216,
             spread=1.0, x="bf16", inf=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _size(rng, lo, hi):
    """_log, and half the time a multiple of 64 where there is room for one."""
    k = _log(rng, lo, hi)
    return max(64, k // 64 * 64) if hi >= 64 and rng.random() < 0.5 else k


def draw(rng):
    op = rng.choice(("ln", "ce", "grad"))
    x = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op == "ln":
        n = _size(rng, 16, 16384)
        rows = _log(rng, 1, min(65536, (1 << 27) // n))
        return dict(op="ln", dir=rng.choice(("fwd", "bwd", "train")), rows=rows, n=n, x=x,
                    p=rng.choice((x, "f32")), pad=rng.choice((0, 0, 1, 8)))
    if op == "ce":
        d = _size(rng, 64, 4096)
        t = _log(rng, 1, 8192)
        v = _size(rng, 256, max(256, min(131072, (1 << 41) // (d * t))))
        return dict(op="ce", dir=rng.choice(("fwd", "train", "train")), t=t, d=d, v=v,
                    x=rng.choice(("bf16", "bf16", "f16")), red=rng.choice(("mean", "sum", "none")),
                    pad=rng.choice((0, 0, 1, 8)))
    count = _log(rng, 1, 400)
    return dict(op="grad", dir=rng.choice(("norm", "clip")), count=count,
                size=_log(rng, 1, min(1 << 24, (1 << 29) // count)),
                spread=rng.choice((1.0, 10.0, 1000.0)), x=x, inf=rng.random() < 0.2)


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def _uniform(g, lo, hi, *shape):
    return lo + (hi - lo) * torch.rand(shape, generator=g, device=DEV)


def _rows_of(t, pad):
    """`t` as a view of a matrix whose rows are `pad` elements longer."""
    if not pad:
        return t
    wide = torch.zeros((t.shape[0], t.shape[1] + pad), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def _sizes(case):
    """Elements of each gradient: case["size"], or spread over a range below it by its logarithm
    (the first one is the largest)."""
    if case["spread"] == 1.0:
        return [case["size"]] * case["count"]
    r = torch.rand(case["count"], generator=torch.Generator().manual_seed(case["count"])).tolist()
    r[0] = 0.0
    return [max(1, int(case["size"] * case["spread"] ** -u)) for u in r]


def prepare(case, seed):
    g = _gen(seed)
    x_type = TYPES[case["x"]]
    if case["op"] == "ln":
        rows, n, p_type = case["rows"], case["n"], TYPES[case["p"]]
        # activations whose columns differ in scale, some of them off zero
        scale = torch.exp(_randn(g, n))
        x = ((_randn(g, rows, n) + 0.3 * _randn(g, n)) * scale).to(x_type)
        s = dict(case=case, x=_rows_of(x, case["pad"]), weight=(1 + 0.1 * _randn(g, n)).to(p_type),
                 bias=(0.1 * _randn(g, n)).to(p_type))
        if case["dir"] != "fwd":
            dy = 10 ** _uniform(g, -2.0, 0.0, rows, 1) * _randn(g, rows, n)
            s["dy"] = _rows_of(dy.to(x_type), case["pad"])
        if case["dir"] == "bwd":        # what the forward pass has left
            xd = x.double()
            mean = xd.mean(1)
            var = (xd - mean[:, None]).square().mean(1)
            s["mean"], s["rstd"] = mean.float(), (var + EPS).rsqrt().float()
        return s
    if case["op"] == "ce":
        t, d, v = case["t"], case["d"], case["v"]
        w = (_randn(g, v, d) * d ** -0.5).to(x_type)
        # frequent words are more frequent, and the network has learned some of them
        target = (v ** torch.rand((t,), generator=g, device=DEV, dtype=torch.float64)).long()
        target = (target - 1).clamp(0, v - 1)
        h = _randn(g, t, d) + _uniform(g, 0.0, 12.0, t, 1) * w[target].float()
        # prompts and padding do not count
        target[torch.rand((t,), generator=g, device=DEV) < 0.1] = IGNORE
        s = dict(case=case, h=_rows_of(h.to(x_type), case["pad"]), w=_rows_of(w, case["pad"]),
                 target=target)
        if case["red"] == "none":
            s["dloss"] = _uniform(g, 0.2, 2.0, t) * (512.0 if x_type == torch.float16 else 1.0 / t)
        else:
            s["dloss"] = torch.full((1,), 1.0 if case["red"] == "sum" else 1024.0, device=DEV)
        return s
    sizes = _sizes(case)
    flat = torch.empty(sum(sizes), dtype=x_type, device=DEV)
    out = torch.empty_like(flat) if case["dir"] == "clip" else flat[:0]
    for part, size in zip(flat.split(sizes), sizes):
        part.normal_(0.0, 1e-2 / (1 + size % 7), generator=g)
    return dict(case=case, grads=list(flat.split(sizes)), flat=out,
                out=list(out.split(sizes)) if case["dir"] == "clip" else None,
                max_norm=1.0, norm_type=math.inf if case["inf"] else 2.0)


# ------------------------------------------------------------------------- the package's calls


def _own(s):
    import unbiased_nvfp4_gradient_amd as nv

    c = s["case"]
    if c["op"] == "ln":
        if c["dir"] == "bwd":
            b = nv.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"],
                                       bias=True)
            return [b.dx, b.dweight, b.dbias]
        f = nv.layer_norm_forward(s["x"], s["weight"], s["bias"], eps=EPS)
        if c["dir"] == "fwd":
            return [f.y, f.mean, f.rstd]
        b = nv.layer_norm_backward(s["dy"], s["x"], f.mean, f.rstd, s["weight"], bias=True)
        return [f.y, b.dx, b.dweight, b.dbias]
    if c["op"] == "ce":
        f = nv.linear_cross_entropy_forward(s["h"], s["w"], s["target"], ignore_index=IGNORE,
                                            reduction=c["red"])
        if c["dir"] == "fwd":
            return [f.loss, f.lse]
        b = nv.linear_cross_entropy_backward(s["dloss"], s["h"], s["w"], s["target"], f.lse,
                                             ignore_index=IGNORE, reduction=c["red"])
        return [f.loss, b.dh, b.dw]
    if c["dir"] == "norm":
        return [nv.grad_norm(s["grads"], norm_type=s["norm_type"])]
    norm = nv.clip_grads(s["grads"], s["max_norm"], norm_type=s["norm_type"], out=s["out"])
    return [norm, s["flat"]]


# ------------------------------------------------------------------------------ the plain forms


def _plain_ln_forward(x, weight, bias):
    xf = x.float()
    mean = xf.mean(1)
    xc = xf - mean[:, None]
    rstd = torch.rsqrt(xc.square().mean(1) + EPS)
    y = xc * rstd[:, None] * weight.float() + bias.float()
    return y.to(x.dtype), mean, rstd


def _plain_ln_backward(dy, x, mean, rstd, weight):
    dyf = dy.float()
    xhat = (x.float() - mean[:, None]) * rstd[:, None]
    g = dyf * weight.float()
    dx = rstd[:, None] * (g - g.mean(1, keepdim=True) - xhat * (g * xhat).mean(1, keepdim=True))
    return (dx.to(x.dtype), (dyf * xhat).sum(0).to(weight.dtype), dyf.sum(0).to(weight.dtype))


def _plain_ce(s, train):
    c, h, w, target = s["case"], s["h"].float(), s["w"].float(), s["target"]
    valid = target != IGNORE
    at = target.clamp(min=0)[:, None]
    logits = h @ w.T
    top = logits.max(1).values
    lse = top + torch.log(torch.exp(logits - top[:, None]).sum(1))
    loss = torch.where(valid, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse))
    left = torch.where(valid, lse, torch.zeros_like(lse))   # tokens that do not count have none
    share = valid.float() * s["dloss"]
    if c["red"] != "none":
        loss = loss.double().sum().float().reshape(1)
    if c["red"] == "mean":
        count = valid.sum().clamp(min=1)
        loss, share = loss / count, share / count
    if not train:
        return [loss, left]
    p = torch.exp(logits - lse[:, None])
    p.scatter_add_(1, at, torch.full_like(at, -1, dtype=p.dtype))
    p *= share[:, None]
    return [loss, (p @ w).to(s["h"].dtype), (p.T @ h).to(s["w"].dtype)]


def _plain_norm(s):
    if math.isinf(s["norm_type"]):
        return torch.stack([t.abs().max() for t in s["grads"]]).max().float().reshape(1)
    sums = torch.stack([t.double().square().sum() for t in s["grads"]])
    return sums.sum().sqrt().float().reshape(1)


def _plain(s):
    c = s["case"]
    if c["op"] == "ln":
        if c["dir"] == "bwd":
            return list(_plain_ln_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"]))
        y, mean, rstd = _plain_ln_forward(s["x"], s["weight"], s["bias"])
        if c["dir"] == "fwd":
            return [y, mean, rstd]
        return [y, *_plain_ln_backward(s["dy"], s["x"], mean, rstd, s["weight"])]
    if c["op"] == "ce":
        return _plain_ce(s, c["dir"] == "train")
    norm = _plain_norm(s)
    if c["dir"] == "norm":
        return [norm]
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    return [norm, torch.cat([(t.float() * coef).to(t.dtype) for t in s["grads"]])]


def run(state):
    return _own(state) if own else _plain(state)


# --------------------------------------------------------------------------- work and exactness


def work(case):
    b = TYPES[case["x"]].itemsize
    if case["op"] == "ln":
        e, n, p = case["rows"] * case["n"], case["n"], TYPES[case["p"]].itemsize
        stats = 8 * case["rows"]
        fwd = 2 * e * b + 2 * n * p + stats, 8 * e
        bwd = 3 * e * b + 3 * n * p + stats, 14 * e
        if case["dir"] != "train":
            by, fl = fwd if case["dir"] == "fwd" else bwd
        else:   # x and dy read once, y and dx written once
            by, fl = 4 * e * b + 4 * n * p, fwd[1] + bwd[1]
        return {"bytes": by, "flops": fl}
    if case["op"] == "ce":
        t, d, v = case["t"], case["d"], case["v"]
        kept = 0.9 * t               # a tenth of the tokens do not count
        by, fl = (kept + v) * d * b + 16 * t, (2 * d + 4) * kept * v
        if case["dir"] == "train":   # and the two products of the gradients
            by, fl = (kept + t + 2 * v) * d * b + 12 * t, (6 * d + 8) * kept * v
        return {"bytes": by, "flops": fl}
    e = sum(_sizes(case))
    if case["dir"] == "norm":
        return {"bytes": e * b + 4, "flops": 2 * e}
    return {"bytes": 2 * e * b + 4, "flops": 3 * e}


def _exact_ln(s):
    c, x = s["case"], s["x"].double()
    n = x.shape[1]
    out = []
    weight = s["weight"].double()
    if c["dir"] == "bwd":
        mean, rstd = s["mean"].double(), s["rstd"].double()
    else:
        mean = x.sum(1) / n
        rstd = 1.0 / torch.sqrt(((x - mean[:, None]) ** 2).sum(1) / n + EPS)
    z = (x - mean[:, None]) * rstd[:, None]
    if c["dir"] != "bwd":
        out.append(z * weight + s["bias"].double())
        if c["dir"] == "fwd":
            return out + [mean, rstd]
    dy = s["dy"].double()
    dz = dy * weight
    # the Jacobian of z: rstd (I - 1 1^T / n - z z^T / n)
    along_one = dz.sum(1, keepdim=True) / n
    along_z = (dz * z).sum(1, keepdim=True) / n
    out.append((dz - along_one - along_z * z) * rstd[:, None])
    return out + [torch.einsum("rn,rn->n", dy, z), dy.sum(0)]


def _exact_ce(s):
    c = s["case"]
    h, w, target = s["h"].double(), s["w"].double(), s["target"]
    t = h.shape[0]
    keep = (target != IGNORE).double()
    scale = 1.0 / max(1.0, float(keep.sum())) if c["red"] == "mean" else 1.0
    loss, lse, dh, dw = [], [], [], torch.zeros_like(w)
    for a in range(0, t, 1024):     # tokens in pieces: 64-bit logits are large
        hb, yb, kb = h[a:a + 1024], target[a:a + 1024].clamp(min=0), keep[a:a + 1024]
        z = torch.matmul(hb, w.t())
        lz = torch.logsumexp(z, 1)
        lse.append(kb * lz)
        rows = torch.arange(len(yb), device=z.device)
        loss.append(kb * (lz - z[rows, yb]))
        if c["dir"] != "train":
            continue
        q = torch.softmax(z, 1)
        q[rows, yb] -= 1.0
        up = s["dloss"].double()
        q *= (kb * scale * (up[a:a + 1024] if c["red"] == "none" else up))[:, None]
        dh.append(torch.matmul(q, w))
        dw += torch.matmul(q.t(), hb)
    loss, lse = torch.cat(loss), torch.cat(lse)
    if c["red"] != "none":
        loss = (loss.sum() * scale).reshape(1)
    return [loss, torch.cat(dh), dw] if c["dir"] == "train" else [loss, lse]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ln":
        return _exact_ln(s)
    if case["op"] == "ce":
        return _exact_ce(s)
    parts = torch.tensor([float(torch.linalg.vector_norm(t, s["norm_type"], dtype=torch.float64))
                          for t in s["grads"]], dtype=torch.float64, device=DEV)
    norm = torch.linalg.vector_norm(parts, s["norm_type"]).reshape(1)
    if case["dir"] == "norm":
        return [norm]
    factor = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    return [norm, torch.cat([factor * t.double() for t in s["grads"]])]
