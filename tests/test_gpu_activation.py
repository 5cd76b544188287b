"""The backward pass of activations and gating on the GPU against 64 bits.

Tolerances count roundings: U = 2^-24 is half a step of float32, HALF[t] half a step of type t."""
import math

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from activation_ref import U, exact, within

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in HALF}   # least subnormal
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KINDS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def strided(t, pad):
    """t as a view into a wider matrix whose other elements are NaN, starting at `pad % 2`."""
    wide = torch.full((t.shape[0], t.shape[1] + 2 * pad), float("nan"), dtype=t.dtype, device=DEV)
    wide[:, pad % 2:pad % 2 + t.shape[1]] = t
    return wide[:, pad % 2:pad % 2 + t.shape[1]]


def check(rows, n, kind, x_type, gated, bias=True, bias_type=None, pad=0, scale=2.0):
    print(f"case: activation backward {rows}x{n} {kind} {x_type} gated={gated} bias={bias} "
          f"pad={pad}", flush=True)
    g = gen(rows * 7 + n)
    wide = (2 if gated else 1) * n
    dy = strided(randn(g, rows, n).to(x_type), pad) if pad else randn(g, rows, n).to(x_type)
    z = (scale * randn(g, rows, wide)).to(x_type)
    z = strided(z, pad + 1) if pad else z
    call = nv.gated_activation_backward if gated else nv.activation_backward
    got = call(dy, z, kind, bias=bias, bias_type=bias_type)
    d = dy.double()
    value, slope, value_tol, slope_tol = exact(z[:, :n], kind)
    if gated:
        up = z[:, n:].double()
        ref = torch.cat([d * up * slope, d * value], 1)
        tol = torch.cat([(d * up).abs() * (slope_tol + 2 * U * slope.abs()),
                         d.abs() * (value_tol + U * value.abs())], 1)
    else:
        ref, tol = d * slope, d.abs() * (slope_tol + U * slope.abs())
    assert got.dz.shape == ref.shape and got.dz.dtype == x_type
    within(got.dz, ref, HALF[x_type] * (ref.abs() + tol) + tol + TINY[x_type], "dz")
    if not bias:
        assert got.dbias is None
        return
    out = bias_type or x_type
    # a lane's rows (of few rows all over 32 lanes, else at most all / 64 and 8), the workgroup's row
    # lanes (at most 256), the partial rows over four parts
    k = rows // 32 + 256 + 512 + 8
    size = ref.abs().sum(0)
    slack = tol.sum(0) + k * U * size
    total = ref.sum(0)
    assert got.dbias.dtype == out
    within(got.dbias, total, HALF[out] * (total.abs() + slack) + slack + TINY[out], "dbias")


@pytest.mark.parametrize("x_type", [F32, BF16, F16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,n", [(1, 1), (3, 7), (257, 1000), (33, 513), (1030, 64)])
def test_activation_backward(rows, n, kind, gated, x_type):
    check(rows, n, kind, x_type, gated)


@pytest.mark.parametrize("rows,n", [(100000, 1), (5000, 9), (70000, 24), (2, 40001), (700, 2048),
                                    (4099, 1023), (1, 16384), (511, 30), (512, 4100), (513, 100)])
@pytest.mark.parametrize("gated,kind", [(False, "gelu"), (True, "silu")])
def test_shapes(rows, n, gated, kind):
    check(rows, n, kind, BF16, gated, bias_type=F32)


@pytest.mark.parametrize("x_type", [F32, BF16, F16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("rows,n,pad", [(7, 1023, 3), (130, 250, 1), (6, 64, 8)])
def test_strides(rows, n, pad, gated, x_type):
    check(rows, n, "gelu_tanh", x_type, gated, pad=pad)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("gated", [False, True])
def test_wide_range(kind, gated):
    # where exponentials overflow and vanish
    check(64, 512, kind, F32, gated, bias=False, scale=60.0)


def test_without_rows_and_without_z():
    dy = torch.zeros(0, 40, device=DEV)
    got = nv.activation_backward(dy, dy, "gelu", bias=True)
    assert got.dz.shape == (0, 40) and torch.equal(got.dbias, torch.zeros(40, device=DEV))
    dy = torch.randn(3, 5, 40, device=DEV).to(BF16)
    got = nv.activation_backward(dy, None, bias=True, bias_type=F32)
    assert torch.equal(got.dz, dy) and got.dz.data_ptr() != dy.data_ptr()
    within(got.dbias, dy.double().sum((0, 1)), 40 * U * dy.double().abs().sum((0, 1)), "dbias")


def test_what_is_not_finite():
    inf, nan = float("inf"), float("nan")
    z = torch.tensor([[-inf, inf, nan, 1e30, -1e30, 0.0, -0.0]], device=DEV)
    dy = torch.ones_like(z)
    for kind in ("gelu", "gelu_tanh", "silu"):
        dz = nv.activation_backward(dy, z, kind).dz[0].tolist()
        assert dz[0] == 0 and dz[1] == 1 and math.isnan(dz[2]) and dz[3] == 1 and dz[4] == 0
        assert dz[5] == dz[6] == 0.5
    dz = nv.activation_backward(dy, z, "relu").dz[0].tolist()
    assert dz == [0, 1, 1, 1, 0, 0, 0]
    # a relu's mask holds whatever the gradient there
    bad = torch.tensor([[inf, nan, nan, 2.0, -inf, nan, inf]], device=DEV)
    dz = nv.activation_backward(bad, z, "relu").dz[0].tolist()
    assert dz[0] == dz[4] == dz[5] == dz[6] == 0 and math.isnan(dz[1]) and dz[3] == 2
    both = torch.cat([z, torch.full_like(z, 3.0)], 1)
    dgate = nv.gated_activation_backward(bad, both, "relu").dz[0, :7].tolist()
    assert dgate[0] == dgate[4] == dgate[5] == dgate[6] == 0
    assert math.isnan(dgate[1]) and dgate[3] == 6


@pytest.mark.parametrize("kind", KINDS)
def test_slopes_against_differences(kind):
    """dz against differences of the activation in 64 bits, away from the relu's corner."""
    z = torch.linspace(-8, 8, 4001, device=DEV, dtype=torch.float64)
    z = z[(z.abs() > 1e-3)].float()
    h = 1e-5
    F = torch.nn.functional
    act = {"none": lambda t: t, "relu": F.relu, "gelu": F.gelu, "silu": F.silu,
           "gelu_tanh": lambda t: F.gelu(t, approximate="tanh")}[kind]
    zd = z.double()
    diff = (act(zd + h) - act(zd - h)) / (2 * h)
    dz = nv.activation_backward(torch.ones_like(z)[None], z[None], kind).dz[0]
    # h^2 / 6 of a third derivative below 3, the differences' own cancellation, the slope's roundings
    within(dz, diff, 1e-10 + 1e-9 + 40 * U, kind)


def test_stream_graph_and_guards():
    g = gen(4)
    rows, n = 1001, 333
    dy, z = randn(g, rows, n).to(BF16), randn(g, rows, 2 * n).to(BF16)
    ref = nv.gated_activation_backward(dy, z, "silu", bias=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nv.gated_activation_backward(dy, z, "silu", bias=True, stream=side)
    side.synchronize()
    assert torch.equal(got.dz, ref.dz) and torch.equal(got.dbias, ref.dbias)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = nv.gated_activation_backward(dy, z, "silu", bias=True)
    for k in range(3):
        dy.copy_(randn(g, rows, n))
        graph.replay()
        torch.cuda.synchronize()
        ref = nv.gated_activation_backward(dy, z, "silu", bias=True)
        assert torch.equal(got.dz, ref.dz) and torch.equal(got.dbias, ref.dbias)
    # through the C ABI between guard elements, in a workspace that held something else
    from unbiased_nvfp4_gradient_amd import block
    L = block._lib()

    def guarded(count, dtype):
        buf = torch.full((count + 128,), 7, dtype=dtype, device=DEV)
        return buf, buf[64:64 + count]
    need = L.activation_backward_workspace_bytes(1, 1, rows, n)
    dz, db, ws = guarded(rows * 2 * n, BF16), guarded(2 * n, F32), guarded(need, torch.uint8)
    assert L.activation_backward(1, 0, 4, 1, dy.data_ptr(), n, z.data_ptr(), 2 * n, rows, n,
                                 dz[1].data_ptr(), db[1].data_ptr(), ws[1].data_ptr(), need,
                                 torch.cuda.current_stream().cuda_stream) == 0
    for buf, inner in (dz, db, ws):
        assert bool((buf[:64] == 7).all()) and bool((buf[-64:] == 7).all())
    assert torch.equal(dz[1].view(rows, 2 * n), ref.dz)


def test_refusals():
    dy = torch.zeros(4, 8, device=DEV)
    with pytest.raises(ValueError, match="z must have the shape"):
        nv.activation_backward(dy, torch.zeros(4, 9, device=DEV), "gelu")
    with pytest.raises(ValueError, match="z must have the shape"):
        nv.gated_activation_backward(dy, dy, "silu")
    with pytest.raises(ValueError, match="z must be a device tensor of float32"):
        nv.activation_backward(dy, dy.to(BF16), "gelu")
    with pytest.raises(ValueError, match="z is needed"):
        nv.activation_backward(dy, None, "gelu")
    with pytest.raises(ValueError, match="bias_type"):
        nv.activation_backward(dy, dy, "gelu", bias=True, bias_type=BF16)
    with pytest.raises(ValueError, match="must be contiguous"):
        nv.activation_backward(torch.zeros(8, 4, device=DEV).t(), dy, "gelu")
