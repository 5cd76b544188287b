"""Edges of the feed-forward block's operators on the GPU: the widest rows and the largest outputs,
sums that are exact, what a type's last values do."""
import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("x_type,rows,n", [(F32, 1, (1 << 29) + 1001), (F32, 2, (1 << 29) - 31),
                                           (BF16, 2, (1 << 30) + 1001)])
def test_activation_backward_of_the_widest_rows(x_type, rows, n):
    """More columns than a launch has threads for: relu's dz exactly, dbias of up to two rows."""
    print(f"case: activation backward {rows}x{n} {x_type}", flush=True)
    g = torch.Generator(device=DEV).manual_seed(n)
    dy = torch.randn((rows, n), generator=g, device=DEV, dtype=x_type)
    z = torch.randn((rows, n), generator=g, device=DEV, dtype=x_type)
    got = nv.activation_backward(dy, z, "relu", bias=True, bias_type=F32)
    dy.masked_fill_(z <= 0, 0)
    assert torch.equal(got.dz, dy)
    total = dy[0].float()
    if rows == 2:
        total += dy[1].float()
    assert torch.equal(got.dbias, total)


@pytest.mark.parametrize("x_type,bits", [(F32, -1), (F32, 0x7FFFFFFF), (F32, -(1 << 23) + 1),
                                         (BF16, -1), (BF16, 0x7FFF), (F16, -1), (F16, 0x7FFF)])
def test_8_bit_moments_of_any_nan(x_type, bits):
    """A gradient that is not a number, whatever its sign and its other bits, makes both moments of its
    block that, and of no other block."""
    print(f"case: adamw 8 bits, a NaN of the bits {bits} of {x_type}", flush=True)
    n = 5 * 128
    p = torch.ones(n, device=DEV, dtype=x_type)
    gr = torch.full((n,), 1e-3, device=DEV, dtype=x_type)
    whole = torch.int32 if x_type is F32 else torch.int16
    gr.view(whole)[300] = bits
    assert bool(gr[300].isnan())
    s = nv.adamw_state(p, 8)
    nv.adamw_step([p], [gr], [s], step=1, lr=1e-3)
    bad = torch.arange(5, device=DEV) == 300 // 128
    for codes, scales, second in ((s.m, s.m_scale, False), (s.v, s.v_scale, True)):
        nan = nv.moment_values(codes, scales, second=second).isnan()
        assert torch.equal(nan.all(1), bad) and torch.equal(nan.any(1), bad), second
    assert p.isnan().nonzero().tolist() == [[300]]


def gradients(seed, n, steps, spread):
    """Normal gradients whose elements' scales are spread below 1, the first of each block 1."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    scale = spread ** -torch.rand(n, generator=g, device=DEV)
    scale[::128] = 1
    for _ in range(steps):
        yield torch.randn(n, generator=g, device=DEV) * scale


@pytest.mark.parametrize("b2", [0.95, 0.999])
@pytest.mark.parametrize("spread", [1e4, 1e6, 1e12])
def test_updates_with_8_bit_moments_are_bounded(spread, b2):
    """AdamW with moments in 8 bits where the elements of a block differ widely.

    With 32 bits an update of such gradients is below 1.4 lr, and so is the largest m of a block against
    its r (both corrected).  The power of two of m's block is at most 2 / 1.875 of its largest m, that of
    r's at least 1 / 1.9375 of its largest r: m's is at most 2.07 * 1.4 = 2.9 of r's.  m's least code is
    2^-17 of the one, r's 2^-18 of the other: where both round to their least, m / r is at most 5.8; rounding
    down to no less than one code takes at most half of r, 2.8 from an m that was 1.4 of it.  8.6 together,
    10 with the gradient's own part."""
    print(f"case: AdamW 8 bits, gradients spread over {spread}, beta2 {b2}", flush=True)
    n, lr = 128 * 512, 1e-3
    p = torch.nn.Parameter(torch.zeros(n, device=DEV))
    opt = nv.AdamW([p], lr=lr, betas=(0.9, b2), eps=1e-8, weight_decay=0.0, bits=8, seed=1)
    worst = torch.zeros((), device=DEV)
    for grad in gradients(7, n, 200, spread):
        before = p.detach().clone()
        p.grad = grad
        opt.step()
        worst = torch.maximum(worst, (p.detach() - before).abs().max())
    assert float(worst) <= 10 * lr, float(worst) / lr


def test_bounded_changes_no_other_code():
    """From one state with and without: the second moment's codes 0 become 1 where it is not 0, and
    nothing else differs."""
    n = 128 * 256
    hyper = dict(lr=1e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1, seed=9)
    p = torch.randn(n, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV)
    s = nv.adamw_state(p, 8)
    changed = 0
    for step, grad in enumerate(gradients(5, n, 4, 1e7), 1):
        grad[torch.arange(n, device=DEV) % 128 > 100] = 0
        q, t = p.clone(), nv.AdamWState(*(None if x is None else x.clone() for x in s))
        r = nv.moment_values(s.v, s.v_scale, second=True).double().view(-1)
        nv.adamw_step([p], [grad], [s], step=step, bounded=True, **hyper)
        nv.adamw_step([q], [grad], [t], step=step, **hyper)
        assert torch.equal(p, q) and torch.equal(s.m, t.m) and torch.equal(s.m_scale, t.m_scale)
        assert torch.equal(s.v_scale, t.v_scale)
        lifted = (t.v.view(-1) == 0) & ((r != 0) | (grad != 0))
        assert torch.equal(s.v.view(-1), torch.where(lifted, 1, t.v.view(-1)))
        changed += int(lifted.sum())
    assert changed > 1000


@pytest.mark.parametrize("b2", [0.95, 0.999])
def test_8_bit_moments_follow_32_bits(b2):
    """200 steps of equal gradients with moments in 8 and in 32 bits.  m moves by much of a code a step:
    its rounding's variance is at most a quarter of the step, (m / 8)^2 / 4, and stays for 1 / (1 - 0.81)
    steps, so that m is off by m / 16 / sqrt(0.19) = 0.15 m.  r leaves its code by (1 - b2) / 2 |g^2 / r^2 -
    1| r a step, which times a code's step r / 16 is the variance of rounding it, and r forgets as much of a
    variance as (1 - b2): off by r sqrt(0.97 / 32) = 0.17 r.  Together 0.23 of the path, which twice that bounds."""
    n, lr = 128 * 512, 1e-3
    p, q = (torch.nn.Parameter(torch.zeros(n, device=DEV)) for _ in range(2))
    a = nv.AdamW([p], lr=lr, betas=(0.9, b2), weight_decay=0.0, bits=8, seed=1)
    b = nv.AdamW([q], lr=lr, betas=(0.9, b2), weight_decay=0.0, bits=32)
    for grad in gradients(11, n, 200, 1e3):
        p.grad = q.grad = grad
        a.step()
        b.step()
    p, q = p.detach().double(), q.detach().double()
    assert float((p - q).norm() / q.norm()) <= 0.5
    # and no drift: the mean difference within six of its spread
    assert abs(float((p - q).mean())) <= 6 * float((p - q).std()) / n ** 0.5


def small(seed, *shape):
    """Whole numbers from -3 to 3."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randint(-3, 4, shape, generator=g, device=DEV, dtype=torch.int8)


@pytest.mark.parametrize("x_type", [F32, BF16, F16])
@pytest.mark.parametrize("rows,n", [(100000, 1), (70000, 24), (5000, 9), (4099, 1023), (513, 100),
                                    (512, 4100), (511, 64), (33, 40001), (7, 300000), (3, 5)])
def test_bias_gradients_count_every_row_once(rows, n, x_type):
    """Small whole numbers, whose sums are exact in float32 in any order."""
    print(f"case: bias gradient {rows}x{n} {x_type}", flush=True)
    dy, z = small(rows, rows, n), small(n, rows, 2 * n)
    got = nv.activation_backward(dy.to(x_type), None, bias=True, bias_type=F32)
    assert torch.equal(got.dz, dy.to(x_type))
    assert torch.equal(got.dbias, dy.double().sum(0).float())
    got = nv.gated_activation_backward(dy.to(x_type), z.to(x_type), "relu", bias=True,
                                       bias_type=F32)
    gate, up = z[:, :n], z[:, n:]
    ref = torch.cat([dy * up * (gate > 0), dy * gate.clamp(min=0)], 1)
    assert torch.equal(got.dz, ref.to(x_type))
    assert torch.equal(got.dbias, ref.double().sum(0).float())


def test_activation_backward_past_31_bits():
    """More than 2^31 elements in dy, 2^32 in dz: dz in its last rows, and every row in dbias."""
    rows, n = 70000, 32771
    print(f"case: gated activation backward {rows}x{n}", flush=True)
    dy, z = small(1, rows, n).to(BF16), small(2, rows, 2 * n).to(BF16)
    got = nv.gated_activation_backward(dy, z, "relu", bias=True, bias_type=F32)
    for at in (slice(0, 3), slice(rows - 40, rows)):
        d, gate, up = dy[at], z[at, :n], z[at, n:]
        ref = torch.cat([d * up * (gate > 0), d * gate.clamp(min=0)], 1)
        assert torch.equal(got.dz[at], ref)
    total = sum(got.dz[k:k + 10000].sum(0, dtype=F32) for k in range(0, rows, 10000))
    assert torch.equal(got.dbias, total)


def operand(seed, rows, k, tiled):
    """An MXFP4 operand of random codes below scales of 1, and a function for the values of its
    rows."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    shape = (k // 128, rows, 64) if tiled else (rows, k // 2)
    codes = torch.randint(0, 256, shape, generator=g, device=DEV, dtype=torch.uint8)
    scales = torch.full((k // 128, rows, 4) if tiled else (rows, k // 32), 127, device=DEV,
                        dtype=torch.uint8)
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device=DEV)

    def values(at):
        c = codes[:, at].transpose(0, 1).flatten(1) if tiled else codes[at]
        return grid[torch.stack([c & 15, c >> 4], 2).flatten(1).int()]
    return nv.MXFP4(codes, scales, tiled), values


@pytest.mark.parametrize("tiled", [True, False])
@pytest.mark.parametrize("rows,n,k,gated", [(65664, 32768, 128, False), (65664, 16387, 256, True),
                                            (65664, 130, 65664, False)])
def test_products_past_31_bits(rows, n, k, gated, tiled):
    """More than 2^31 elements in y and z, or 2^31 bytes in an operand: the first and the last rows.  The
    sums are exact: multiples of a quarter below 2^22."""
    print(f"case: product {rows}x{n}x{k} gated={gated} tiled={tiled}", flush=True)
    a, a_rows = operand(1, rows, k, tiled)
    b, b_rows = operand(2, (1 + gated) * n, k, tiled)
    if gated:
        got = nv.mxfp4_gated_forward(a, b, activation="relu", keep_z=True)
    else:
        got = nv.mxfp4_linear_forward(a, b, activation="relu", keep_z=True)
    w = b_rows(slice(None))
    for at in (slice(0, 70), slice(rows - 300, rows)):
        z = (a_rows(at).double() @ w.double().T).float()
        assert torch.equal(got.z[at], z.to(BF16))
        y = z[:, :n].clamp(min=0) * z[:, n:] if gated else z.clamp(min=0)
        assert torch.equal(got.y[at], y.to(BF16))


@pytest.mark.parametrize("gated", [False, True])
def test_layer_without_gradients_gives_the_same_output(gated):
    from unbiased_nvfp4_gradient_amd.linear import QuartetLinear
    torch.manual_seed(4)
    kw = dict(scheme="sr", scales="mx", activation="silu", gated=gated, bias=True, dtype=BF16,
              device=DEV)
    a, b = QuartetLinear(256, 384, **kw), QuartetLinear(256, 384, **kw)
    b.load_state_dict(a.state_dict())
    x = torch.randn(128, 256, device=DEV).to(BF16)
    with torch.no_grad():
        got = a(x)
    assert torch.equal(got, b(x).detach()) and not got.requires_grad
