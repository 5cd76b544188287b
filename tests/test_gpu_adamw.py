"""AdamW on the GPU against plain 64-bit implementations, and its 8-bit moments code by code.

Tolerances count roundings: U = 2^-24 is half a step of float32, HALF[t] half a step of type t."""
import math

import numpy as np
import pytest
import torch

import oracle
import unbiased_nvfp4_gradient_amd as nv

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in HALF}   # least subnormal
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


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


def make(g, sizes, kind, bits=32, master=False, pad=0):
    """(params, grads, states) of slices of flat buffers, `pad` elements apart, and the buffers:
    NaN everywhere between the slices."""
    def flat(dtype):
        return torch.full((sum(n + pad for n in sizes) + pad,), float("nan"), dtype=dtype,
                          device=DEV)

    def slices(buf):
        out, at = [], pad
        for n in sizes:
            out.append(buf[at:at + n])
            at += n + pad
        return out
    bufs = [flat(kind), flat(kind)] + [flat(F32) for _ in range(3)]
    params, grads, m, v, w = [slices(b) for b in bufs]
    states = []
    for i, n in enumerate(sizes):
        w[i].copy_(0.02 * randn(g, n))
        params[i].copy_(w[i])
        grads[i].copy_(1e-3 * randn(g, n))
        s = nv.AdamWState(m[i], v[i], master=w[i] if master else None)
        m[i].copy_(1e-3 * randn(g, n))
        v[i].copy_(1e-6 * torch.rand(n, generator=g, device=DEV))
        if bits == 8:
            s = nv.adamw_state(params[i], 8)._replace(master=s.master)
        states.append(s)
    return params, grads, states, bufs


def reference(p, g, m, v, step, coef=1.0, lr=0.0, betas=(0.0, 0.0), eps=0.0, weight_decay=0.0):
    """(p, m, v, slack of p, m, v) in 64 bits."""
    b1, b2 = betas
    p, g, m, v = p.double(), g.double() * coef, m.double(), v.double()
    # the gradient's factor has 3 roundings and its product one, each weight and each product one,
    # the sum one; squares double the gradient's
    sm = 8 * U * (b1 * m.abs() + (1 - b1) * g.abs())
    sv = 13 * U * (b2 * v + (1 - b2) * g * g)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    den = (v / (1 - b2 ** step)).sqrt() + eps
    rate = lr / (1 - b1 ** step)
    # den: half of v's 13, then root, sqrt, product, eps and sum; the quotient, rate and product
    sp = 4 * U * p.abs() + rate * (sm / den + (7 + 5 + 3) * U * m.abs() / den)
    p = p * (1 - lr * weight_decay) - rate * m / den
    return p, m, v, sp + 2 * U * p.abs(), sm, sv


SIZES = ((1,), (4099, 1, 3, 128, 0, 2048, 2049, 77777), (1 << 20,))


@pytest.mark.parametrize("kind,master", [(F32, False), (BF16, False), (BF16, True), (F16, False),
                                         (F16, True)])
@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("pad", [0, 1, 5])
def test_adamw(kind, master, sizes, pad):
    print(f"case: adamw {sizes} {kind} master={master} pad={pad}", flush=True)
    g = gen(len(sizes) + pad)
    params, grads, states, bufs = make(g, sizes, kind, master=master, pad=pad)
    old = [b.clone() for b in bufs]
    norm = nv.grad_norm(grads)
    max_norm = 0.5 * float(norm)
    before = [(s.master if master else p).clone() for p, s in zip(params, states)]
    was = [(s.m.clone(), s.v.clone()) for s in states]
    nv.adamw_step(params, grads, states, step=7, norm=norm, max_norm=max_norm, **HYPER)
    coef = max_norm / (float(norm) + 1e-6)
    for p, gr, s, b, (m, v) in zip(params, grads, states, before, was):
        rp, rm, rv, sp, sm, sv = reference(b, gr, m, v, 7, coef, **HYPER)
        within(s.m, rm, sm + TINY[F32], "m")
        within(s.v, rv, sv + TINY[F32], "v")
        if master:
            within(s.master, rp, sp, "master")
            assert torch.equal(p, s.master.to(kind))
        else:
            within(p, rp, HALF[kind] * (rp.abs() + sp) + sp + TINY[kind], "p")
    assert torch.equal(bufs[1].nan_to_num(7.0), old[1].nan_to_num(7.0))      # gradients are read
    for new, was in zip(bufs, old):                                          # between the slices
        assert torch.equal(new.isnan(), was.isnan())


def coded(x, noise, fraction):
    """Codes and scale bytes of float32 [blocks, 128] by the format's definition, in 64 bits."""
    top = np.abs(x).max(1)
    mantissa, e = np.frexp(top.astype(np.float64))                 # top = mantissa 2^e
    steps = np.ceil(mantissa * 2 ** (fraction + 1))                # of a code in [2^(e-1), 2^e]
    e = np.where(steps == 2 ** (fraction + 1), e, e - 1)           # top <= largest code of 2^e
    e = np.where(top == 0, -126, np.maximum(e, -126))
    size = np.abs(x).astype(np.float64)
    own = np.where(size == 0, -10000, np.frexp(size)[1] - 1)       # a zero is a subnormal
    field = np.maximum(own - e[:, None] + 15, 1)                   # exponent field, 1 for subnormals
    unit = np.ldexp(1.0, (e[:, None] + field - 15 - fraction).astype(np.int64))
    count = np.floor(size / unit + noise / 65536.0)                # in steps of the code
    code = np.minimum(count + (field - 1) * 2 ** fraction, 2 ** (fraction + 4) - 1).astype(np.int64)
    if fraction == 3:
        code += 128 * ((x < 0) & (code > 0))
    return code.astype(np.uint8), (e + 127).astype(np.uint8)


def noise_of(seed, tensor, step, blocks):
    i = np.arange(blocks * 32, dtype=np.uint64)
    ctr = np.stack([i & 0xFFFFFFFF, i >> 32, np.full_like(i, (1 << 31) + tensor),
                    np.full_like(i, step & 0xFFFFFFFF)], 1).astype(np.uint32)
    w = oracle.philox_n(np.full(len(i), seed, dtype=np.uint64), ctr).reshape(blocks, 128)
    return (w >> 16).astype(np.float64), (w & 0xFFFF).astype(np.float64)


@pytest.mark.parametrize("kind,master", [(F32, False), (BF16, False), (F16, True)])
@pytest.mark.parametrize("sizes", [(1,), (127, 128, 129), (4097, 0, 5, 70000, 2048)])
@pytest.mark.parametrize("pad", [0, 3])
def test_adamw_8_bits(kind, master, sizes, pad, oracle_mod):
    """Every code and scale of four steps, from float32 arithmetic of one rounding an
    operation; gradients spread over many powers of two, so that codes below the range occur."""
    print(f"case: adamw 8 bits {sizes} {kind} master={master} pad={pad}", flush=True)
    g = gen(sum(sizes) + pad)
    params, grads, states, bufs = make(g, sizes, kind, bits=8, master=master, pad=pad)
    b1, b2 = (np.float32(b) for b in HYPER["betas"])
    c1, c2 = (np.float32(1 - b) for b in HYPER["betas"])
    seed = 0x123456789ABCDEF
    for step in (1, 2, 3, 1 << 33):
        for t in grads:
            t.copy_(1e-3 * randn(g, len(t)) * 10 ** -(6 * torch.rand(len(t), generator=g,
                                                                     device=DEV)))
        was = [(nv.moment_values(s.m, s.m_scale).cpu().numpy(),
                nv.moment_values(s.v, s.v_scale, second=True).cpu().numpy()) for s in states]
        before = [(s.master if master else p).clone() for p, s in zip(params, states)]
        nv.adamw_step(params, grads, states, step=step, seed=seed, **HYPER)
        for k, (p, gr, s, b, (m, r)) in enumerate(zip(params, grads, states, before, was)):
            n, blocks = len(p), len(s.m)
            if n == 0:
                continue
            gg = np.zeros(blocks * 128, dtype=np.float32)
            gg[:n] = gr.float().cpu().numpy()
            gg = gg.reshape(blocks, 128)
            m = b1 * m + c1 * gg
            r = np.sqrt(b2 * (r * r) + c2 * (gg * gg))
            up, low = noise_of(seed, k, step, blocks)
            for what, x, noise, fraction, code, scale in (("m", m, up, 3, s.m, s.m_scale),
                                                          ("r", r, low, 4, s.v, s.v_scale)):
                ref, e = coded(x, noise, fraction)
                assert np.array_equal(scale.cpu().numpy(), e), (what, step, k)
                got = code.cpu().numpy()
                assert np.array_equal(got, ref), (what, step, k, int((got != ref).sum()))
                values = nv.moment_values(code, scale, second=fraction == 4).cpu().numpy()
                mag = (got & 127 if fraction == 3 else got).astype(np.int64)
                f, field = mag % 2 ** fraction, mag >> fraction
                size = np.where(field == 0, f * 2.0, f + 2 ** fraction) * \
                    2.0 ** (field - 15 - fraction + e[:, None].astype(np.int64) - 127)
                if fraction == 3:
                    size = np.where(got > 127, -size, size)
                assert np.array_equal(values, size.astype(np.float32)), (what, step, k)
            m, r = (torch.from_numpy(t.reshape(-1)[:n]).to(DEV) for t in (m, r))
            b1d, b2d = HYPER["betas"]
            den = r.double() / math.sqrt(1 - b2d ** step) + HYPER["eps"]
            rate = HYPER["lr"] / (1 - b1d ** step)
            rp = b.double() * (1 - HYPER["lr"] * HYPER["weight_decay"]) - rate * m.double() / den
            sp = 4 * U * b.double().abs() + 9 * U * rate * m.double().abs() / den \
                + 2 * U * rp.abs()
            if master:
                within(s.master, rp, sp, "master")
                assert torch.equal(p, s.master.to(kind))
            else:
                within(p, rp, HALF[kind] * (rp.abs() + sp) + sp + TINY[kind], "p")
    assert bool(bufs[0][:pad].isnan().all())


def test_8_bit_moments_of_tiny_gradients(oracle_mod):
    """Squares below the range in which the square root's short form holds, subnormal ones, and
    zeros."""
    g = gen(12)
    n, seed = 6 * 128, 77
    p = randn(g, n)
    gr = randn(g, n) * 10.0 ** (-12 - 11 * torch.rand(n, generator=g, device=DEV))
    gr[128:256] *= 1e-16
    gr[300:340] = 0
    gr[512:640] = 0
    s = nv.adamw_state(p, 8)
    nv.adamw_step([p], [gr], [s], step=1, seed=seed, **HYPER)
    gg = gr.cpu().numpy().reshape(6, 128)
    c1, c2 = (np.float32(1 - b) for b in HYPER["betas"])
    up, low = noise_of(seed, 0, 1, 6)
    for what, x, noise, fraction, code, scale in (
            ("m", c1 * gg, up, 3, s.m, s.m_scale),
            ("r", np.sqrt(c2 * (gg * gg)), low, 4, s.v, s.v_scale)):
        ref, e = coded(x, noise, fraction)
        assert np.array_equal(scale.cpu().numpy(), e), what
        assert np.array_equal(code.cpu().numpy(), ref), what


def test_8_bit_moments_of_what_is_not_finite():
    n = 1000
    p = torch.ones(n, device=DEV)
    gr = torch.full((n,), 1e-3, device=DEV)
    gr[130], gr[400], gr[700] = float("nan"), float("inf"), -3e38
    s = nv.adamw_state(p, 8)
    nv.adamw_step([p], [gr], [s], step=1, **HYPER)
    m = nv.moment_values(s.m, s.m_scale)
    r = nv.moment_values(s.v, s.v_scale, second=True)
    bad = torch.zeros(8, dtype=torch.bool, device=DEV)
    bad[[130 // 128, 400 // 128]] = True
    assert torch.equal(m.isnan().all(1), bad) and torch.equal(m.isnan().any(1), bad)
    bad[700 // 128] = True                                   # its square is infinite
    assert torch.equal(r.isnan().all(1), bad) and torch.equal(r.isnan().any(1), bad)
    assert torch.equal(p.isnan().nonzero()[:, 0].cpu(), torch.tensor([130, 400]))
    # the parameter with the infinite square: m / infinity
    assert float(p[700]) == pytest.approx(1 - HYPER["lr"] * HYPER["weight_decay"], rel=4 * U)


@pytest.mark.parametrize("bits", [32, 8])
def test_no_gradient_at_all(bits):
    p = torch.randn(777, device=DEV).to(BF16)
    before = p.clone()
    s = nv.adamw_state(p, bits)
    nv.adamw_step([p], [torch.zeros_like(p)], [s], step=1, **HYPER)
    factor = torch.tensor(1 - HYPER["lr"] * HYPER["weight_decay"], dtype=F32, device=DEV)
    assert torch.equal(p, (before.float() * factor).to(BF16))
    assert not bool(s.m.any()) and not bool(s.v.any())


def test_8_bit_moments_keep_their_mean():
    """A second moment whose gradients stop decays as beta2^t on average, though a step changes it
    by far less than a code's; nearest rounding would keep it for ever."""
    n, steps, b2 = 128 * 256, 400, 0.999
    p = torch.zeros(n, device=DEV)
    s = nv.adamw_state(p, 8)
    hyper = dict(HYPER, betas=(0.9, b2))
    nv.adamw_step([p], [torch.ones_like(p)], [s], step=1, seed=3, **hyper)
    first = float(nv.moment_values(s.v, s.v_scale, second=True).double().mean())
    zero = torch.zeros_like(p)
    for t in range(2, steps + 2):
        nv.adamw_step([p], [zero], [s], step=t, seed=3, **hyper)
    r = nv.moment_values(s.v, s.v_scale, second=True).double()
    # rounding sqrt(v) keeps its mean, and so adds its variance to v: f (1 - f) q^2 a step with
    # f = (1 - sqrt(b2)) r / q of a code's step q <= r / 16, at most (1 - sqrt(b2)) r^2 / 16, a
    # sixteenth of half of what v loses: v decays 31/32 as fast, or faster
    low, high = first * b2 ** (steps / 2), first * b2 ** (steps / 2 * 31 / 32)
    # beside it the mean's own spread over n elements: the variance of one is below steps times the
    # bound above
    spread = 6 * math.sqrt(steps * (1 - math.sqrt(b2)) / 16 / n) * first
    assert low - spread <= float((r ** 2).mean().sqrt()) <= high + spread
    # m: 0.9^400 is 0
    assert float(nv.moment_values(s.m, s.m_scale).abs().max()) < 1e-6


def test_more_tensors_than_a_launch_takes():
    """300 parameters, every third with 8 bits, in one call and one by one: the same bits."""
    g = gen(5)
    sizes = [1 + 37 * k % 5000 for k in range(300)]

    def build():
        gg = gen(9)
        a = make(gg, sizes, BF16, bits=32)
        b = make(gg, sizes, BF16, bits=8)
        pick = [b if k % 3 == 0 else a for k in range(300)]
        return [[pick[k][i][k] for k in range(300)] for i in range(3)]
    params, grads, states = build()
    one, gone, sone = build()
    for t, o in zip(grads, gone):
        t.copy_(1e-3 * randn(g, len(t)))
        o.copy_(t)
    nv.adamw_step(params, grads, states, step=3, seed=11, **HYPER)
    for k in range(300):
        nv.adamw_step([one[k]], [gone[k]], [sone[k]], step=3, seed=11, **HYPER)
    for k in range(300):
        assert torch.equal(params[k], one[k]), k
        for field, x, y in zip(nv.AdamWState._fields, states[k], sone[k]):
            # the noise is by a parameter's place in the list
            if x is not None and (k % 3 or k == 0 or field.endswith("scale")):
                assert torch.equal(x, y), (k, field)
    # equal parameters of one list draw noise of their own
    p = [torch.ones(4096, device=DEV) for _ in range(2)]
    gr = [torch.linspace(0.1, 1, 4096, device=DEV)] * 2
    s = [nv.adamw_state(t, 8) for t in p]
    nv.adamw_step(p, gr, s, step=1, seed=2, **HYPER)
    assert torch.equal(p[0], p[1]) and not torch.equal(s[0].m, s[1].m)


@pytest.mark.parametrize("bits", [32, 8])
def test_graph_follows_step_and_rate(bits):
    """A captured call reads the step and the rate at each replay; its results are the eager
    call's, with other work between the replays."""
    g = gen(2)
    sizes = (5000, 17)
    params, grads, states, _ = make(g, sizes, BF16, bits=bits, master=True)
    eager = [p.clone() for p in params]
    es = [nv.AdamWState(*(None if t is None else t.clone() for t in s)) for s in states]
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    lr = torch.tensor([1e-3], device=DEV)
    hyper = dict(betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, seed=4, max_norm=0.01)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        norm = nv.grad_norm(grads)
        nv.adamw_step(params, grads, states, step=step, lr=lr, norm=norm, **hyper)
    for k in range(1, 5):
        for t in grads:
            t.copy_(1e-2 * randn(g, len(t)))
        rate = float(torch.tensor(1e-3 / k))
        lr.fill_(rate)
        graph.replay()
        torch.cuda.synchronize()
        nv.adamw_step(eager, grads, es, step=k, lr=float(lr), norm=nv.grad_norm(grads), **hyper)
        for p, e, s, x in zip(params, eager, states, es):
            assert torch.equal(p, e)
            assert all(a is None or torch.equal(a, b) for a, b in zip(s, x))


def test_numbers_as_tensors_on_the_host():
    p, q = torch.ones(100, device=DEV), torch.ones(100, device=DEV)
    gr = torch.linspace(-1, 1, 100, device=DEV)
    nv.adamw_step([p], [gr], [nv.adamw_state(p)], step=torch.tensor(3), lr=torch.tensor(0.125))
    nv.adamw_step([q], [gr], [nv.adamw_state(q)], step=3, lr=0.125)
    assert torch.equal(p, q)


def test_other_stream():
    g = gen(8)
    params, grads, states, _ = make(g, (70000,), F32)
    twin = make(gen(8), (70000,), F32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    nv.adamw_step(params, grads, states, step=2, stream=side, **HYPER)
    side.synchronize()
    nv.adamw_step(*twin[:3], step=2, **HYPER)
    assert torch.equal(params[0], twin[0][0]) and torch.equal(states[0].v, twin[2][0].v)


def test_versions_of_written_tensors():
    p, gr = torch.ones(10, device=DEV), torch.ones(10, device=DEV)
    s = nv.adamw_state(p)
    versions = [t._version for t in (p, gr, s.m, s.v)]
    nv.adamw_step([p], [gr], [s], step=1, lr=0.1)
    assert [t._version - v for t, v in zip((p, gr, s.m, s.v), versions)] == [1, 0, 1, 1]


def test_more_elements_than_32_bits_count():
    """2^32 + 2^12 + 5 elements: the last ones as a parameter of their own."""
    n, tail = (1 << 32) + 4096 + 5, 4096 + 5
    print(f"case: adamw {n} bf16, 8 bits", flush=True)
    p = torch.zeros(n, dtype=BF16, device=DEV)
    gr = torch.zeros(n, dtype=BF16, device=DEV)
    g = gen(3)
    p[-tail:] = randn(g, tail).to(BF16)
    gr[-tail:] = (1e-3 * randn(g, tail)).to(BF16)
    s = nv.adamw_state(p, 8)
    q, qs = p[-tail:].clone(), nv.adamw_state(p[-tail:], 8)
    nv.adamw_step([p], [gr], [s], step=1, **HYPER)
    nv.adamw_step([q], [gr[-tail:]], [qs], step=1, **HYPER)
    assert torch.equal(p[-tail:], q) and torch.equal(s.m_scale[-33:], qs.m_scale)
    assert torch.equal(s.v_scale[-33:], qs.v_scale) and not bool(s.m[:-33].any())
    # codes by the noise of their own counters: within a step of each other
    a, b = (nv.moment_values(t, qs.m_scale) for t in (s.m[-33:], qs.m))
    assert bool(((a - b).abs() <= b.abs() / 8 + torch.exp2(qs.m_scale.float() - 127 - 17)[:, None])
                .all())


@pytest.mark.parametrize("bits", [32, 8])
def test_refusals_on_the_device(bits):
    p, gr = torch.ones(300, device=DEV, dtype=BF16), torch.ones(300, device=DEV, dtype=BF16)
    s = nv.adamw_state(p, bits, master=True)

    def refused(match, params=p, grads=gr, state=s, **over):
        with pytest.raises(ValueError, match=match):
            nv.adamw_step([params], [grads], [state], **{**dict(step=1, lr=1e-3), **over})
    refused("grad .* does not fit", grads=gr.float())
    refused("grad .* does not fit", grads=gr[1:])
    refused("contiguous", grads=torch.ones(600, device=DEV, dtype=BF16)[::2])
    refused("v .* does not fit", state=s._replace(v=s.v.reshape(-1)[:-1]))
    refused("v .* does not fit", state=s._replace(v=s.v.half()))
    refused("master .* does not fit", state=s._replace(master=s.master.to(BF16)))
    refused("master .* does not fit", params=p.float(), grads=gr.float())
    refused("v of parameter 0 is missing", state=s._replace(v=None))
    if bits == 8:
        refused("m_scale of parameter 0 is missing", state=tuple(s[:2]))
        refused("v_scale .* does not fit", state=s._replace(v_scale=s.v_scale[:-1]))
    else:
        refused("m_scale .* does not fit", state=s._replace(m_scale=s.m.byte()))
    refused("norm and max_norm", norm=torch.ones(1, device=DEV))
    refused("max_norm must not", norm=torch.ones(1, device=DEV), max_norm=-1.0)
    refused("norm must be", norm=torch.ones(2, device=DEV), max_norm=1.0)
    refused("whole number from 1", step=0)
    refused("step must be", step=torch.ones(1, device=DEV))
    refused("lr must be", lr=torch.ones(1, device=DEV, dtype=torch.float64))
    refused("on one GPU", grads=gr.cpu())
    with pytest.raises(nv.NVFP4Error) as e:
        nv.adamw_step([p, p], [gr, gr], [s, nv.adamw_state(p, bits)], step=1, lr=1e-3)
    assert e.value.status == nv.ERR_ARG
    with pytest.raises(ValueError, match="scales must be"):
        nv.moment_values(torch.zeros(3, 128, dtype=torch.uint8, device=DEV),
                         torch.zeros(2, dtype=torch.uint8, device=DEV))


def test_optimizer_follows_torch():
    """The optimizer against torch's own in float64 over five steps, a parameter without a gradient
    at first, a gradient that is no contiguous tensor, two groups."""
    g = gen(1)
    shapes = [(33, 70), (5,), (64, 64)]
    ours = [torch.nn.Parameter(randn(g, *s)) for s in shapes]
    theirs = [torch.nn.Parameter(p.detach().double()) for p in ours]
    groups = lambda ps: [dict(params=ps[:2], weight_decay=0.3), dict(params=ps[2:], lr=2e-2)]  # noqa: E731
    a = nv.AdamW(groups(ours), lr=1e-2, betas=(0.8, 0.9), eps=1e-6)
    b = torch.optim.AdamW(groups(theirs), lr=1e-2, betas=(0.8, 0.9), eps=1e-6)
    for k in range(5):
        for i, (p, q) in enumerate(zip(ours, theirs)):
            if i == 1 and k < 2:
                continue
            grad = randn(g, *shapes[i][::-1]).t() if len(shapes[i]) == 2 else randn(g, *shapes[i])
            p.grad, q.grad = grad, grad.double()
        a.step()
        b.step()
    # a step moves a parameter by about its rate, off by some 30 roundings of it, and by the
    # parameter's own rounding
    for i, (p, q) in enumerate(zip(ours, theirs)):
        rate = 2e-2 if i == 2 else 1e-2
        within(p.detach(), q.detach(), 5 * U * (6 * q.detach().abs() + 6) + 5 * 60 * U * rate,
               f"parameter {i}")


def test_optimizer_refuses_capture():
    p = torch.nn.Parameter(torch.ones(10, device=DEV))
    p.grad = torch.ones(10, device=DEV)
    opt = nv.AdamW([p])
    scratch = torch.zeros(4, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        scratch += 1
        with pytest.raises(RuntimeError, match="on the host"):
            opt.step()
    assert not opt.state


def test_resumed_training_is_the_same():
    x = [torch.sin(torch.arange(1000, device=DEV) * float(k + 1)).to(BF16) for k in range(6)]
    start = torch.randn(1000, device=DEV).to(BF16)

    def run(p, opt, grads):
        for t in grads:
            p.grad = t
            opt.step(norm=nv.grad_norm([p.grad]), max_norm=1.0)
    p = torch.nn.Parameter(start.clone())
    opt = nv.AdamW([p], lr=1e-2, bits=8, master=True, seed=5)
    run(p, opt, x)
    q = torch.nn.Parameter(start.clone())
    first = nv.AdamW([q], lr=1e-2, bits=8, master=True, seed=5)
    run(q, first, x[:3])
    second = nv.AdamW([q], lr=7.0)
    second.load_state_dict(first.state_dict())
    run(q, second, x[3:])
    assert torch.equal(p, q)
    for k, t in opt.state[p].items():
        assert t == 6 if k == "step" else torch.equal(t, second.state[q][k])
