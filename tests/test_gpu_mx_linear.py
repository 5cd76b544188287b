"""Products of MXFP4 operands with their epilogue (bias, activation, residual, gating) on the GPU
against 64 bits.

Tolerances count roundings: U = 2^-24 is half a step of float32, HALF[t] half a step of type t.  A sum
of K exact products in FP32 is off by at most K U times the sum of their magnitudes."""
import ctypes

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from activation_ref import U, exact, within
from unbiased_nvfp4_gradient_amd import block

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
TINY = {t: torch.finfo(t).smallest_normal * torch.finfo(t).eps for t in HALF}   # least subnormal
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
KINDS = ("none", "relu", "gelu", "gelu_tanh", "silu")
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SLOPE = 1.13            # above every activation's largest slope


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def operand(g, rows, k, spread=3, tiled=False, scale=0):
    """(MXFP4, its values in 64 bits): random codes below block scales of 2^(scale - spread) and
    up."""
    codes = torch.randint(0, 256, (rows, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    e = torch.randint(scale - spread, scale + 1, (rows, k // 32), generator=g, device=DEV)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=DEV)
    x = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], 2).view(rows, k)
    x = (x.view(rows, k // 32, 32) * torch.exp2(e.double())[:, :, None]).view(rows, k)
    scales = (e + 127).to(torch.uint8)
    if tiled:
        codes = codes.view(rows, k // 128, 64).transpose(0, 1).contiguous()
        scales = scales.view(rows, k // 128, 4).transpose(0, 1).contiguous()
    return nv.MXFP4(codes, scales, tiled), x


def check(m, n, k, kind="none", dtype=BF16, gated=False, bias=None, residual=None, tiled=True,
          rotated=False, keep_z=True, seed=0):
    """`bias` a type, `residual` a number of elements between its rows."""
    print(f"case: mx linear {m}x{n}x{k} {kind} {dtype} gated={gated} bias={bias} "
          f"residual={residual} tiled={tiled}", flush=True)
    g = gen(seed + m * 31 + n * 7 + k)
    wide = 2 * n if gated else n
    # values of about 1 after the product
    a, av = operand(g, m, k, tiled=tiled, scale=7 if rotated else 0)
    b, bv = operand(g, wide, k, tiled=tiled, scale=-int(k).bit_length() // 2 - 2)
    b_vec = randn(g, wide).to(bias) if bias else None
    res = None
    if residual is not None:
        res = torch.full((m, n + residual), float("nan"), dtype=dtype, device=DEV)
        res[:, :n] = randn(g, m, n)
        res = res[:, :n]
    call = dict(bias=b_vec, activation=kind, rotated_pair=rotated, dtype=dtype, keep_z=keep_z)
    if gated:
        got = nv.mxfp4_gated_forward(a, b, **call)
    else:
        got = nv.mxfp4_linear_forward(a, b, residual=res, **call)
    f = 2.0 ** -7 if rotated else 1.0
    z = f * torch.matmul(av, bv.t().contiguous())
    dz = k * U * f * torch.matmul(av.abs(), bv.abs().t().contiguous())
    if b_vec is not None:
        z = z + b_vec.double()
        dz = dz + U * z.abs()
    value, _, value_tol, _ = exact(z[:, :n], kind)
    tol = value_tol + SLOPE * dz[:, :n]
    if gated:
        up = z[:, n:]
        ref = value * up
        tol = tol * (up.abs() + dz[:, n:]) + value.abs() * dz[:, n:] + U * ref.abs()
    else:
        ref = value
        if res is not None:
            ref = ref + res.double()
            tol = tol + U * ref.abs()
    assert got.y.shape == (m, n) and got.y.dtype == dtype
    tol = 1.01 * tol
    within(got.y, ref, HALF[dtype] * (ref.abs() + tol) + tol + TINY[dtype], "y")
    if not keep_z:
        assert got.z is None
        return
    assert got.z.shape == (m, wide) and got.z.dtype == dtype
    dz = 1.01 * dz
    within(got.z, z, HALF[dtype] * (z.abs() + dz) + dz + TINY[dtype], "z")


# one row and more than a kernel for few rows takes, tiles of 128 and of 256 that end inside, one column
SHAPES = [(1, 1, 128), (1, 8192, 256), (3, 70, 384), (31, 129, 640), (32, 64, 2048), (33, 65, 128),
          (64, 200, 512), (65, 7, 1152), (127, 128, 256), (130, 257, 384), (257, 255, 128),
          (300, 1000, 640), (1000, 300, 128), (520, 2100, 384), (1300, 1500, 128),
          (1030, 1101, 2176)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_shapes(m, n, k, tiled, gated):
    check(m, n, k, "gelu", BF16, gated, bias=F32, residual=None if gated else 3, tiled=tiled)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m,n,k", [(5, 77, 512), (200, 99, 256)])
def test_activations_and_types(m, n, k, kind, gated, dtype):
    check(m, n, k, kind, dtype, gated, bias=dtype, residual=None if gated else 0, rotated=True,
          keep_z=kind != "relu")


@pytest.mark.parametrize("m", [1, 33, 140])
@pytest.mark.parametrize("bias", [None, F32, F16])
@pytest.mark.parametrize("residual", [None, 0, 1, 8])
def test_with_and_without(m, bias, residual):
    check(m, 75, 256, "silu", F16, bias=bias, residual=residual)


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("k", [128, 256, 384, 1024])
def test_tiles_of_256(k, tiled, gated):
    # more than there are compute units, so that some take a second tile, the last ones cut; fewer steps
    # of K than are in flight, and more
    check(4090, 2200 if gated else 4399, k, "silu", BF16, gated, tiled=tiled)


# 200 tiles of 256, fewer than compute units, and 190; the least K that takes tiles of 256, and less
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m,k,tiled", [(2500, 4096, True), (2500, 3968, True), (2500, 2048, False),
                                       (2500, 1920, False), (2400, 2048, False)])
def test_almost_enough_tiles_of_256(m, k, tiled, gated):
    n = 4900 if m == 2500 else 4801
    check(m, n // 2 if gated else n, k, "silu", BF16, gated, bias=BF16, tiled=tiled)


@pytest.mark.parametrize("dtype", [F32, F16])
@pytest.mark.parametrize("k", [128, 512])
def test_several_tiles_of_128_a_workgroup(k, dtype):
    check(3900, 3700, k, "none", dtype, residual=1, bias=F32)


def test_outputs_that_pass_by_the_caches():
    check(16500, 8195, 128, "relu", BF16, bias=F32)
    check(16500, 4099, 128, "silu", BF16, gated=True)


@pytest.mark.parametrize("m,n,k", [(0, 5, 128), (5, 0, 128), (0, 0, 0)])
def test_empty(m, n, k):
    a, _ = operand(gen(1), m, max(k, 128))
    b, _ = operand(gen(2), n, max(k, 128))
    got = nv.mxfp4_linear_forward(a, b, keep_z=True)
    assert got.y.shape == got.z.shape == (m, n)


@pytest.mark.parametrize("gated", [False, True])
def test_no_elements_to_sum_over(gated):
    a = nv.empty_mx_layout(5, 0, DEV)
    b = nv.empty_mx_layout(14, 0, DEV)
    bias = torch.linspace(-2, 2, 14, device=DEV)
    call = nv.mxfp4_gated_forward if gated else nv.mxfp4_linear_forward
    got = call(a, b, bias=bias, activation="relu", dtype=F32, keep_z=True)
    ref = bias.expand(5, 14)
    assert torch.equal(got.z, ref)
    value = ref.clamp(min=0)
    assert torch.equal(got.y, value[:, :7] * ref[:, 7:] if gated else value)


def test_same_product_as_the_gemm():
    """Without an epilogue, the bits of mxfp4_gemm's result (more rows than the kernel for few takes)."""
    for m, n, k, tiled in ((256, 512, 1024, True), (96, 160, 512, False), (4096, 4096, 256, True)):
        a, _ = operand(gen(m), m, k, tiled=tiled)
        b, _ = operand(gen(n), n, k, tiled=tiled)
        got = nv.mxfp4_linear_forward(a, b, rotated_pair=True, dtype=F32)
        assert torch.equal(got.y, nv.mxfp4_gemm(a, b, rotated_pair=True))


def test_wide_scales():
    """Block scales over many powers of two, and the byte for NaN."""
    for m in (4, 300):
        check(m, 130, 512, seed=m)
        g = gen(m)
        a, av = operand(g, m, 256, spread=60, scale=30)
        b, bv = operand(g, 70, 256, spread=60, scale=30)
        got = nv.mxfp4_linear_forward(a, b, dtype=F32).y
        ref = torch.matmul(av, bv.t().contiguous())
        size = torch.matmul(av.abs(), bv.abs().t().contiguous())
        within(got, ref, 256 * U * size + U * ref.abs(), "wide scales")
        a.scales.view(-1, 4)[0, 0] = 255
        got = nv.mxfp4_linear_forward(a, b, dtype=F32).y
        assert bool(got[0].isnan().all()) and not bool(got[1:].isnan().any())


def test_what_is_not_finite():
    for m in (3, 200):
        a, _ = operand(gen(m), m, 128)
        b, _ = operand(gen(m + 1), 40, 128)
        bias = torch.zeros(40, device=DEV)
        bias[3], bias[5], bias[7] = float("nan"), float("inf"), float("-inf")
        res = torch.zeros(m, 40, device=DEV)
        res[1, 11] = float("nan")
        y = nv.mxfp4_linear_forward(a, b, bias=bias, activation="relu", residual=res, dtype=F32).y
        assert bool(y[:, 3].isnan().all()) and bool((y[:, 5] == float("inf")).all())
        assert bool((y[:, 7] == 0).all())
        bad = y.isnan()
        assert bool(bad[1, 11]) and int(bad.sum()) == m + 1


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("m", [1, 7, 150])
def test_stream_graph_and_repeat(m, gated):
    g = gen(m)
    a, _ = operand(g, m, 1024)
    b, _ = operand(g, 600, 1024)
    other, _ = operand(g, m, 1024)
    call = nv.mxfp4_gated_forward if gated else nv.mxfp4_linear_forward
    ref = call(a, b, activation="silu", keep_z=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = call(a, b, activation="silu", keep_z=True, stream=side)
    side.synchronize()
    assert torch.equal(got.y, ref.y) and torch.equal(got.z, ref.z)
    graphs = []
    for x in (a, other):                      # two graphs of the same calls, replayed in turns
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = call(x, b, activation="silu", keep_z=True)
        graphs.append((graph, out, call(x, b, activation="silu", keep_z=True)))
    for _ in range(3):
        for graph, _, _ in graphs:
            graph.replay()
        call(other, b, activation="gelu")
        torch.cuda.synchronize()
        for _, out, want in graphs:
            assert torch.equal(out.y, want.y) and torch.equal(out.z, want.z)


@pytest.mark.parametrize("m,n,k,gated", [(1, 333, 512, 0), (9, 77, 2048, 1), (40, 129, 128, 0),
                                         (131, 259, 256, 1), (1100, 1030, 256, 0),
                                         (1100, 1030, 256, 1)])
@pytest.mark.parametrize("tiled", [0, 1])
def test_guards(m, n, k, gated, tiled):
    """Outputs between guard elements, through the C ABI."""
    L = block._lib()
    wide = 2 * n if gated else n
    a, _ = operand(gen(m), m, k, tiled=bool(tiled))
    b, _ = operand(gen(n), wide, k, tiled=bool(tiled))

    def guarded(count, dtype):
        buf = torch.full((count + 512,), 7, dtype=dtype, device=DEV)
        return buf, buf[256:256 + count]
    y, z = guarded(m * n, BF16), guarded(m * wide, BF16)
    assert L.mxfp4_linear_forward(nv._cmx(a), nv._cmx(b), m, n, k, 0, gated, 4, 1, 1, None, None, 0,
                                  y[1].data_ptr(), z[1].data_ptr(),
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    for buf, _ in (y, z):
        assert bool((buf[:256] == 7).all()) and bool((buf[-256:] == 7).all())
    call = nv.mxfp4_gated_forward if gated else nv.mxfp4_linear_forward
    ref = call(a, b, activation="silu", keep_z=True)
    assert torch.equal(y[1].view(m, n), ref.y) and torch.equal(z[1].view(m, wide), ref.z)


def test_refusals():
    a, b = nv.empty_mx_layout(4, 256, DEV), nv.empty_mx_layout(6, 256, DEV)

    def refused(match, x=a, w=b, call=nv.mxfp4_linear_forward, **over):
        with pytest.raises(ValueError, match=match):
            call(x, w, **over)
    refused("unknown activation", activation="tanh")
    refused("dtype must be", dtype=torch.float64)
    refused("both K-tiled", w=nv.empty_mx_layout(6, 256, DEV, k_tiled=True))
    refused("b.codes must be", w=nv.empty_mx_layout(6, 128, DEV))
    refused("multiple of 128", x=nv.empty_mx_layout(4, 64, DEV), w=nv.empty_mx_layout(6, 64, DEV))
    refused("for the gate", w=nv.empty_mx_layout(7, 256, DEV), call=nv.mxfp4_gated_forward)
    refused("bias must be", bias=torch.zeros(5, device=DEV))
    refused("bias must be", bias=torch.zeros(6, device=DEV, dtype=F16))
    refused("bias must be", bias=torch.zeros(3, device=DEV), call=nv.mxfp4_gated_forward)
    refused("residual must have", residual=torch.zeros(4, 5, device=DEV, dtype=BF16))
    refused("residual must be", residual=torch.zeros(4, 6, device=DEV))
    refused("contiguous", residual=torch.zeros(6, 4, device=DEV, dtype=BF16).t())
    refused("must be on a GPU", x=nv.empty_mx_layout(4, 256, "cpu"))
