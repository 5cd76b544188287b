"""Cases for timing the operators of a feed-forward block on MXFP4 operands and of its update: the
FP4 product with bias, activation and residual in its epilogue, the gated product (both
projections, the activation and their product), the activations' backward passes with the bias
gradient, and AdamW over many tensors with moments in 32 or 8 bits.

`run` computes a case in its plain form (elementary torch operations in 32 bits, rounded once
at the end) or, where `own` is true, with this package's kernels; `exact` gives the same
results from the definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")
BETAS, EPS = (0.9, 0.95), 1e-8
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)       # E2M1
BLOCK = 128                                            # elements of an 8-bit moment's block


def listed():
    return [
        # one token through a feed-forward layer's first matrix while generating: latency
        dict(name="linear 1x8192x2048 bf16 gelu", op="linear", m=1, n=8192, k=2048, y="bf16",
             act="gelu_tanh", bias=True, res=False, z=False, tiled=True, rot=True, pad=0),
        # odd rows and columns, row-major operands, a residual that is a view, float16
        dict(name="linear 1537x5003x2176 f16", op="linear", m=1537, n=5003, k=2176, y="f16",
             act="none", bias=True, res=True, z=False, tiled=False, rot=False, pad=5),
        # the second matrix of a feed-forward layer and the residual stream, a short batch
        dict(name="linear 2048x2048x8192 bf16 res", op="linear", m=2048, n=2048, k=8192,
             y="bf16", act="none", bias=False, res=True, z=False, tiled=True, rot=True, pad=0),
        # the repository's largest product; the pre-activation is kept for the backward pass
        dict(name="linear 16384x8192x8192 bf16", op="linear", m=16384, n=8192, k=8192, y="bf16",
             act="gelu", bias=True, res=False, z=True, tiled=True, rot=True, pad=0),
        # a few sequences that each produce one token, gate and up projection
        dict(name="gated 7x8192x2048 bf16 silu", op="gated", m=7, n=8192, k=2048, y="bf16",
             act="silu", bias=False, z=False, tiled=True, rot=True),
        # the 1.9B model's gate and up projections in training (32768 tokens, 2048 -> 8192)
        dict(name="gated 32768x8192x2048 bf16", op="gated", m=32768, n=8192, k=2048, y="bf16",
             act="silu", bias=False, z=True, tiled=True, rot=True),
        # a small batch in float32: latency
        dict(name="act bwd 257x1000 f32 gelu", op="act", rows=257, n=1000, x="f32", act="gelu",
             gated=False, bias=True, pad=0),
        # that model's gated block backwards
        dict(name="gated bwd 32768x8192 bf16", op="act", rows=32768, n=8192, x="bf16", act="silu",
             gated=True, bias=True, pad=0),
        # the parameters of one small layer: latency
        dict(name="adamw 9x4099 f32", op="adamw", count=9, size=4099, spread=1.0, x="f32",
             bits=32, master=False, clip=False, step=1),
        # large bfloat16 matrices with float32 masters, clipped by the norm of their gradients
        dict(name="adamw 48x8388608 bf16 master", op="adamw", count=48, size=8388608, spread=1.0,
             x="bf16", bits=32, master=True, clip=True, step=1000),
        # many tensors of very different sizes, moments in 8 bits
        dict(name="adamw 300x40001 f32 8 bits", op="adamw", count=300, size=40001, spread=100.0,
             x="f32", bits=8, master=False, clip=True, step=20),
        # large matrices, moments in 8 bits
        dict(name="adamw 24x4194304 bf16 8 bits", op="adamw", count=24, size=4194304, spread=1.0,
             x="bf16", bits=8, master=False, clip=False, step=5000),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def _size(rng, lo, hi):
    """_log, and half the time a multiple of 64 where there is room for one."""
    k = _log(rng, lo, hi)
    return max(64, k // 64 * 64) if hi >= 64 and rng.random() < 0.5 else k


def draw(rng):
    op = rng.choice(("linear", "linear", "gated", "act", "adamw", "adamw"))
    y = rng.choice(("bf16", "bf16", "f16", "f32"))
    if op in ("linear", "gated"):
        k = 128 * _log(rng, 1, 64)
        n = _size(rng, 16, 8192)
        m = _log(rng, 1, 16384)
        case = dict(op=op, m=m, n=n, k=k, y=y, act=rng.choice(ACTIVATIONS),
                    bias=rng.random() < 0.5, z=rng.random() < 0.4, tiled=rng.random() < 0.7,
                    rot=rng.random() < 0.5)
        if op == "linear":
            case.update(res=rng.random() < 0.5, pad=rng.choice((0, 0, 1, 8)))
        return case
    if op == "act":
        n = _size(rng, 16, 16384)
        return dict(op=op, rows=_log(rng, 1, min(65536, (1 << 27) // n)), n=n, x=y,
                    act=rng.choice(ACTIVATIONS), gated=rng.random() < 0.5,
                    bias=rng.random() < 0.7, pad=rng.choice((0, 0, 1, 8)))
    count = _log(rng, 1, 400)
    return dict(op=op, count=count, size=_log(rng, 1, min(1 << 23, (1 << 26) // count)),
                spread=rng.choice((1.0, 10.0, 1000.0)), x=y, bits=rng.choice((32, 8)),
                master=y != "f32" and rng.random() < 0.5, clip=rng.random() < 0.5,
                step=_log(rng, 1, 100000))


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 31)


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


def _to_mx(x, tiled):
    """(codes, scales) of a float32 matrix: one power of two per 32 elements of a row, the
    smallest that lets 6 cover them, and E2M1 codes to nearest; K-tiled where asked for."""
    rows, k = x.shape
    blocks = x.view(rows, k // 32, 32)
    e = torch.ceil(torch.log2(blocks.abs().amax(2) / 6)).clamp(-127, 127)
    size = (blocks * torch.exp2(-e)[:, :, None]).abs()
    mag = torch.zeros(size.shape, dtype=torch.uint8, device=x.device)
    for lo, hi in zip(GRID[:-1], GRID[1:]):
        mag += size > (lo + hi) / 2
    codes = (mag + 8 * (blocks < 0).to(torch.uint8)).view(rows, k // 2, 2)
    codes, scales = codes[:, :, 0] | codes[:, :, 1] << 4, (e + 127).to(torch.uint8)
    if tiled:
        codes = codes.view(rows, k // 128, 64).transpose(0, 1)
        scales = scales.view(rows, k // 128, 4).transpose(0, 1)
    return codes.contiguous(), scales.contiguous()


def _sizes(case):
    """Elements of each parameter: case["size"], or spread over a range below it by its logarithm
    (the first one is the largest)."""
    if case["spread"] == 1.0:
        return [case["size"]] * case["count"]
    r = torch.rand(case["count"], generator=torch.Generator().manual_seed(case["count"])).tolist()
    r[0] = 0.0
    return [max(1, int(case["size"] * case["spread"] ** -u)) for u in r]


def _prepare_product(case, g):
    m, k, gated = case["m"], case["k"], case["op"] == "gated"
    n = (2 if gated else 1) * case["n"]
    y_type = TYPES[case["y"]]
    # activations whose columns differ in scale; a rotated pair's product is 128 times the plain one
    a = _randn(g, m, k) * torch.exp(0.5 * _randn(g, k)) * (128.0 if case["rot"] else 1.0)
    w = _randn(g, n, k) * k ** -0.5
    s = dict(case=case, a=_to_mx(a, case["tiled"]), b=_to_mx(w, case["tiled"]), bias=None,
             residual=None)
    if case["bias"]:
        s["bias"] = (0.3 * _randn(g, n)).to(torch.float32 if n % 2 else y_type)
    if case.get("res"):
        s["residual"] = _rows_of(_randn(g, m, n).to(y_type), case["pad"])
    return s


def _prepare_act(case, g):
    rows, n, x_type = case["rows"], case["n"], TYPES[case["x"]]
    dy = 10 ** _uniform(g, -2.0, 0.0, rows, 1) * _randn(g, rows, n)
    z = 2 * _randn(g, rows, (2 if case["gated"] else 1) * n) + 0.3 * _randn(g, 1, 1)
    return dict(case=case, dy=_rows_of(dy.to(x_type), case["pad"]),
                z=_rows_of(z.to(x_type), case["pad"]))


def _prepare_adamw(case, g):
    """Parameters, gradients and moments as slices of flat buffers (8-bit moments: of a buffer
    of blocks, the last one of each parameter padded with zeros)."""
    sizes, x_type = _sizes(case), TYPES[case["x"]]
    total = sum(sizes)
    s = dict(case=case, p=(0.02 * _randn(g, total)).to(x_type),
             g=torch.empty(total, dtype=x_type, device=DEV), lr=3e-4, decay=0.1, seed=case["step"])
    for part, size in zip(s["g"].split(sizes), sizes):
        part.normal_(0.0, 1e-3 / (1 + size % 7), generator=g)
    master = s["p"].float() + 1e-5 * _randn(g, total) if case["master"] else None
    if master is not None:
        s["p"] = master.to(x_type)
    m, r = 3e-4 * _randn(g, total), 6e-4 * _uniform(g, 0.3, 1.5, total)
    s["norm"] = (1e-3 * total ** 0.5 * (1 + torch.rand(1, generator=g, device=DEV)))
    s["max_norm"] = 0.7e-3 * total ** 0.5 if case["clip"] else None
    s["params"], s["grads"] = list(s["p"].split(sizes)), list(s["g"].split(sizes))
    s["master"] = master
    masters = list(master.split(sizes)) if master is not None else [None] * len(sizes)
    if case["bits"] == 32:
        s["m"], s["v"] = m, r.square()
        s["moments"] = [(a, b, None, None, c) for a, b, c in
                        zip(s["m"].split(sizes), s["v"].split(sizes), masters)]
        return s
    # elements of every parameter's blocks in the flat order; past a parameter's end: `total`
    count = torch.tensor([-(-n // BLOCK) for n in sizes], device=DEV)
    ends = torch.tensor(sizes, device=DEV).cumsum(0)
    of = torch.repeat_interleave(torch.arange(len(sizes), device=DEV), count)
    first = count.cumsum(0) - count
    start = ends[of] - torch.tensor(sizes, device=DEV)[of] \
        + BLOCK * (torch.arange(len(of), device=DEV) - first[of])
    at = start[:, None] + torch.arange(BLOCK, device=DEV)
    s["at"] = torch.where(at < ends[of][:, None], at, torch.full_like(at, total))
    s["group"] = (at - start[:, None] + BLOCK * (torch.arange(len(of), device=DEV)
                                                 - first[of])[:, None])[:, ::4] // 4
    s["tensor"] = of
    grid = [torch.cat([t, t.new_zeros(1)])[s["at"]] for t in (m, r)]
    half = [torch.full_like(t, 1 << 15, dtype=torch.int32) for t in grid]
    s["m8"], s["m_scale"] = _encode(grid[0], half[0], 3)
    s["r8"], s["r_scale"] = _encode(grid[1], half[1], 4)
    counts = count.tolist()
    s["moments"] = list(zip(s["m8"].split(counts), s["r8"].split(counts),
                            s["m_scale"].split(counts), s["r_scale"].split(counts), masters))
    return s


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] in ("linear", "gated"):
        return _prepare_product(case, g)
    return _prepare_act(case, g) if case["op"] == "act" else _prepare_adamw(case, g)


# ------------------------------------------------------------------------- the package's calls


def _own(s):
    import unbiased_nvfp4_gradient_amd as nv

    c = s["case"]
    if c["op"] in ("linear", "gated"):
        a, b = nv.MXFP4(*s["a"], c["tiled"]), nv.MXFP4(*s["b"], c["tiled"])
        if c["op"] == "gated":
            f = nv.mxfp4_gated_forward(a, b, bias=s["bias"], activation=c["act"],
                                       rotated_pair=c["rot"], dtype=TYPES[c["y"]], keep_z=c["z"])
        else:
            f = nv.mxfp4_linear_forward(a, b, bias=s["bias"], activation=c["act"],
                                        residual=s["residual"], rotated_pair=c["rot"],
                                        dtype=TYPES[c["y"]], keep_z=c["z"])
        return [f.y, f.z] if c["z"] else [f.y]
    if c["op"] == "act":
        call = nv.gated_activation_backward if c["gated"] else nv.activation_backward
        b = call(s["dy"], s["z"], c["act"], bias=c["bias"])
        return [b.dz, b.dbias] if c["bias"] else [b.dz]
    nv.adamw_step(s["params"], s["grads"], s["moments"], step=c["step"], lr=s["lr"], betas=BETAS,
                  eps=EPS, weight_decay=s["decay"], norm=s["norm"] if c["clip"] else None,
                  max_norm=s["max_norm"], seed=s["seed"])
    out = [s["p"]] + ([s["master"]] if c["master"] else [])
    if c["bits"] == 32:
        return out + [s["m"], s["v"]]
    return out + [nv.moment_values(s["m8"], s["m_scale"]),
                  nv.moment_values(s["r8"], s["r_scale"], second=True)]


# ------------------------------------------------------------------------------ the plain forms


def _values(codes, scales, tiled):
    """The float32 matrix that MXFP4 codes and scales stand for."""
    if tiled:
        codes = codes.transpose(0, 1).reshape(codes.shape[1], -1)
        scales = scales.transpose(0, 1).reshape(scales.shape[1], -1)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), device=codes.device)
    pairs = torch.stack([codes & 15, codes >> 4], 2).view(codes.shape[0], -1)
    x = grid[pairs.int()].view(codes.shape[0], -1, 32)
    return (x * torch.exp2(scales.float() - 127)[:, :, None]).view(codes.shape[0], -1)


def _activation(z, kind):
    if kind == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if kind == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z)) if kind == "silu" else z


def _slope(z, kind):
    """The activation's derivative."""
    if kind == "relu":
        return (z > 0).to(z.dtype)
    if kind == "gelu":
        cdf = 0.5 * (1 + torch.erf(z * math.sqrt(0.5)))
        return cdf + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if kind == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    if kind == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    return torch.ones_like(z)


def _plain_product(s):
    c, y_type = s["case"], TYPES[s["case"]["y"]]
    z = _values(*s["a"], c["tiled"]) @ _values(*s["b"], c["tiled"]).T
    if c["rot"]:
        z *= 2.0 ** -7
    if s["bias"] is not None:
        z += s["bias"].float()
    if c["op"] == "gated":
        y = _activation(z[:, :c["n"]], c["act"]) * z[:, c["n"]:]
    else:
        y = _activation(z, c["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
    return [y.to(y_type), z.to(y_type)] if c["z"] else [y.to(y_type)]


def _plain_act(s):
    c, dy, z = s["case"], s["dy"].float(), s["z"].float()
    if c["gated"]:
        gate, up = z[:, :c["n"]], z[:, c["n"]:]
        dz = torch.cat([dy * up * _slope(gate, c["act"]), dy * _activation(gate, c["act"])], 1)
    else:
        dz = dy * _slope(z, c["act"])
    x_type = s["dy"].dtype
    return [dz.to(x_type), dz.sum(0).to(x_type)] if c["bias"] else [dz.to(x_type)]


def _power(e):
    """2^e of whole numbers -126..127, exactly."""
    return ((e + 127).int() << 23).view(torch.float32)


def _encode(x, noise, mantissa):
    """Blocks of float32 as 8-bit floating codes of four exponent and `mantissa` bits (with three,
    bit 7 is the sign) below one power of two each, rounded by 16-bit noise."""
    cut = 23 - mantissa
    top = x.abs().amax(1).view(torch.int32)
    scale = (((top + (1 << cut) - 1) >> 23)).clamp(1, 254)
    t = x.abs() * _power((127 - scale).clamp(-126, 127))[:, None] * 2.0 ** -112
    code = ((t.view(torch.int32) + (noise << (cut - 16))) >> cut).clamp(max=(16 << mantissa) - 1)
    if mantissa == 3:
        code = code + ((x < 0) & (code > 0)).int() * 128
    return code.to(torch.uint8), scale.to(torch.uint8)


def _decode(code, scale, mantissa):
    """The float32 values of _encode's codes."""
    mag = code & 127 if mantissa == 3 else code
    x = (mag.int() << (23 - mantissa)).view(torch.float32) * 2.0 ** 112
    x = x * _power((scale.int() - 127).clamp(-126, 127))[:, None]
    return torch.where(code > 127, -x, x) if mantissa == 3 else x


def _high(a, b):
    """The upper 32 bits of the product of a (below 2^32, in 64 bits) and a 32-bit number."""
    return ((a >> 16) * b + ((a & 0xFFFF) * b >> 16)) >> 16


def _noise(s, step):
    """Two 16-bit random numbers for each element of every block: Philox4x32-10 of the key
    `seed` at (group of four elements, 0, 2^31 + tensor, step); an element's word gives its first
    moment's in the upper and its second moment's in the lower half."""
    word = 0xFFFFFFFF
    a = s["group"]
    b = torch.zeros_like(a)
    c = torch.broadcast_to((s["tensor"] + (1 << 31))[:, None], a.shape)
    d = torch.full_like(a, step & word)
    k0, k1 = s["seed"] & word, s["seed"] >> 32 & word
    for _ in range(10):
        a, b, c, d = (_high(c, 0xCD9E8D57) ^ b ^ k0, c * 0xCD9E8D57 & word,
                      _high(a, 0xD2511F53) ^ d ^ k1, a * 0xD2511F53 & word)
        k0, k1 = k0 + 0x9E3779B9 & word, k1 + 0xBB67AE85 & word
    w = torch.stack([a, b, c, d], 2).view(a.shape[0], BLOCK)
    return (w >> 16).int(), (w & 0xFFFF).int()


def _plain_adamw(s):
    c = s["case"]
    b1, b2 = BETAS
    c1, c2 = 1 - b1 ** c["step"], 1 - b2 ** c["step"]
    grad = s["g"].float()
    if c["clip"]:
        factor = torch.full_like(s["norm"], s["max_norm"]) / (s["norm"] + 1e-6)
        grad = grad * factor.clamp(max=1.0)
    if c["bits"] == 8:
        grid = lambda t: torch.cat([t, t.new_zeros(1)])[s["at"]]  # noqa: E731
        gg = grid(grad)
        m = b1 * _decode(s["m8"], s["m_scale"], 3) + (1 - b1) * gg
        r = _decode(s["r8"], s["r_scale"], 4)
        r = torch.sqrt(b2 * (r * r) + (1 - b2) * (gg * gg))
        up, low = _noise(s, c["step"])
        for at, new in zip(("m8", "m_scale", "r8", "r_scale"),
                           _encode(m, up, 3) + _encode(r, low, 4)):
            s[at].copy_(new)
        inside = s["at"] < s["p"].numel()
        m, root = m[inside], r[inside]
    else:
        m = b1 * s["m"] + (1 - b1) * grad
        v = b2 * s["v"] + (1 - b2) * (grad * grad)
        s["m"].copy_(m)
        s["v"].copy_(v)
        root = torch.sqrt(v)
    p = s["master"] if c["master"] else s["p"].float()
    p = p * (1 - s["lr"] * s["decay"]) - s["lr"] / c1 * (m / (root / math.sqrt(c2) + EPS))
    s["p"].copy_(p)
    out = [s["p"]]
    if c["master"]:
        s["master"].copy_(p)
        out.append(s["master"])
    if c["bits"] == 32:
        return out + [s["m"], s["v"]]
    return out + [_decode(s["m8"], s["m_scale"], 3), _decode(s["r8"], s["r_scale"], 4)]


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    if op in ("linear", "gated"):
        return _plain_product(state)
    return _plain_act(state) if op == "act" else _plain_adamw(state)


# --------------------------------------------------------------------------- work and exactness


def work(case):
    if case["op"] in ("linear", "gated"):
        m, n, k, b = case["m"], case["n"], case["k"], TYPES[case["y"]].itemsize
        wide = 2 * n if case["op"] == "gated" else n
        by = (m + wide) * k * 17 / 32 + m * n * b + case["z"] * m * wide * b
        by += case.get("res", False) * m * n * b + case["bias"] * 4 * wide
        return {"bytes": by, "flops": 2 * m * wide * k + 10 * m * n}
    if case["op"] == "act":
        e, b = case["rows"] * case["n"], TYPES[case["x"]].itemsize
        wide = 2 if case["gated"] else 1
        return {"bytes": e * b * (1 + 2 * wide), "flops": (10 + 4 * wide) * e}
    e, b = sum(_sizes(case)), TYPES[case["x"]].itemsize
    by = e * (b + b + (8 if case["master"] else b))     # gradient, parameter written, and read
    if case["bits"] == 32:
        return {"bytes": by + 16 * e, "flops": 16 * e}
    # codes read and written; the values that they stand for are given back in 32 bits
    return {"bytes": by + 4 * e + 8 * e, "flops": 60 * e}


def _exact_values(codes, scales, tiled):
    if tiled:
        codes, scales = (torch.cat(list(t.unbind(0)), 1) for t in (codes, scales))
    even, odd = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    x = torch.stack([even, odd], -1).flatten(1)
    sign = 1.0 - 2.0 * (x >= 8)
    mag = x % 8
    # subnormals 0 and 1/2, then (1 + half) 2^(exponent - 1)
    e, half = torch.floor(mag / 2), mag % 2
    size = torch.where(e == 0, half / 2, (1 + half / 2) * 2.0 ** (e - 1))
    return sign * size * (2.0 ** (scales.double() - 127)).repeat_interleave(32, 1)


def _exact_activation(z, kind):
    """(value, derivative)."""
    F = torch.nn.functional
    with torch.enable_grad():
        x = z.detach().clone().requires_grad_()
        y = {"none": lambda t: t * 1.0, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
             "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[kind](x)
        slope, = torch.autograd.grad(y.sum(), x)
    return y.detach(), slope


def _exact_product(s):
    c = s["case"]
    w = _exact_values(*s["b"], c["tiled"])
    a = _exact_values(*s["a"], c["tiled"])
    if c["rot"]:
        a /= 128.0
    ys, zs = [], []
    for at in range(0, c["m"], 4096):        # tokens in pieces: 64-bit matrices are large
        z = torch.mm(a[at:at + 4096], w.t())
        if s["bias"] is not None:
            z += s["bias"].double()
        if c["op"] == "gated":
            y = _exact_activation(z[:, :c["n"]], c["act"])[0] * z[:, c["n"]:]
        else:
            y = _exact_activation(z, c["act"])[0]
            if s["residual"] is not None:
                y += s["residual"][at:at + 4096].double()
        ys.append(y)
        if c["z"]:
            zs.append(z)
    return [torch.cat(ys), torch.cat(zs)] if c["z"] else [torch.cat(ys)]


def _exact_act(s):
    c, dy, z = s["case"], s["dy"].double(), s["z"].double()
    if c["gated"]:
        value, slope = _exact_activation(z[:, :c["n"]], c["act"])
        dz = torch.hstack([slope * z[:, c["n"]:] * dy, value * dy])
    else:
        dz = _exact_activation(z, c["act"])[1] * dy
    return [dz, torch.mv(dz.t(), torch.ones_like(dz[:, 0]))] if c["bias"] else [dz]


def _exact_adamw(s):
    """8-bit moments have no value here: which of two codes noise rounds to hangs on the last bit
    of the 32-bit number."""
    c = s["case"]
    b1, b2 = BETAS
    grad = s["g"].double()
    if c["clip"]:
        grad *= min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
    if c["bits"] == 8:
        inside = s["at"] < s["p"].numel()
        block = s["m_scale"].double()[:, None] - 127
        sign, mag = 1.0 - 2.0 * (s["m8"] >= 128), (s["m8"] % 128).double()
        e, f = torch.floor(mag / 8), mag % 8 / 8
        m = sign * torch.where(e == 0, f * 2, 1 + f) * 2.0 ** (e - 15 + block)
        block, mag = s["r_scale"].double()[:, None] - 127, s["r8"].double()
        e, f = torch.floor(mag / 16), mag % 16 / 16
        r = torch.where(e == 0, f * 2, 1 + f) * 2.0 ** (e - 15 + block)
        m, v = m[inside], r[inside] ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = m + (1 - b1) * (grad - m)
    v = v + (1 - b2) * (grad ** 2 - v)
    p = (s["master"] if c["master"] else s["p"]).double()
    p = p - s["lr"] * s["decay"] * p
    p -= s["lr"] * (m / (1 - b1 ** c["step"])) / ((v / (1 - b2 ** c["step"])).sqrt() + EPS)
    out = [p, p] if c["master"] else [p]
    return out + ([m, v] if c["bits"] == 32 else [None, None])


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("linear", "gated"):
        return _exact_product(s)
    return _exact_act(s) if case["op"] == "act" else _exact_adamw(s)
