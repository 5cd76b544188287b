"""The feed-forward block's operators and AdamW as a training step uses them: linear layers on the
MXFP4 recipe with bias, activation, residual and gating, and the whole step of a small model."""
import importlib.util
import os

import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from activation_ref import U, exact, within
from unbiased_nvfp4_gradient_amd import linear
from unbiased_nvfp4_gradient_amd.linear import EpilogueLinearFunction, QuartetLinear

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
HALF = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.bfloat16, torch.float16)}
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SLOPE = 1.13            # above every activation's largest slope


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def values(q):
    """The 64-bit matrix that a K-tiled MXFP4 operand stands for."""
    codes = q.codes.transpose(0, 1).reshape(q.codes.shape[1], -1)
    scales = q.scales.transpose(0, 1).reshape(q.scales.shape[1], -1)
    grid = torch.tensor(GRID + tuple(-v for v in GRID), dtype=torch.float64, device=DEV)
    x = torch.stack([grid[(codes & 15).long()], grid[(codes >> 4).long()]], 2)
    x = x.view(codes.shape[0], -1, 32) * torch.exp2(scales.double() - 127)[:, :, None]
    return x.view(codes.shape[0], -1)


def product(a, b):
    """(A B^T of a rotated pair, a bound of its FP32 sum's error) in 64 bits."""
    x, y = values(a), values(b)
    k = x.shape[1]
    return 2.0 ** -7 * (x @ y.t().contiguous()), \
        2.0 ** -7 * k * U * (x.abs() @ y.abs().t().contiguous())


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("kind,gated,bias,residual", [
    ("none", False, False, True), ("none", False, True, False), ("gelu", False, True, True),
    ("silu", True, True, False), ("relu", True, False, False)])
def test_layer(kind, gated, bias, residual, dtype):
    """Output and every gradient against the formulas on the layer's own operands."""
    print(f"case: layer {kind} gated={gated} bias={bias} residual={residual} {dtype}", flush=True)
    g = gen(3)
    T, inn, out, seed = 256, 384, 128, 5
    wide = 2 * out if gated else out
    x = randn(g, T, inn).to(BF16).requires_grad_()
    w = (randn(g, wide, inn) * inn ** -0.5).to(BF16).requires_grad_()
    b = (0.3 * randn(g, wide)).requires_grad_() if bias else None
    r = randn(g, T, out).to(dtype).requires_grad_() if residual else None
    y = EpilogueLinearFunction.apply(x, w, b, r, seed, "sr", kind, gated, dtype)
    dy = randn(g, T, out).to(dtype)
    y.backward(dy)
    qx = linear._quantize("rtn", x.detach(), 0, 2 * seed, ("row",), "mx").row
    qw = linear._quantize("rtn", w.detach(), 0, 2 * seed, ("row",), "mx").row
    z, dz_tol = product(qx, qw)
    if bias:
        z = z + b.detach().double()
        dz_tol = dz_tol + U * z.abs()
    value, _, tol, _ = exact(z[:, :out], kind)
    tol = tol + SLOPE * dz_tol[:, :out]
    ref = value
    if gated:
        up = z[:, out:]
        ref = value * up
        tol = tol * (up.abs() + dz_tol[:, out:]) + value.abs() * dz_tol[:, out:] + U * ref.abs()
    if residual:
        ref = ref + r.detach().double()
        tol = tol + U * ref.abs()
        assert torch.equal(r.grad, dy)
    assert y.dtype == dtype
    within(y.detach(), ref, HALF[dtype] * (ref.abs() + tol) + 1.01 * tol, "y")
    # dz as the layer forms it, from z as it was kept; then its products
    kept = (nv.mxfp4_gated_forward if gated else nv.mxfp4_linear_forward)(
        qx, qw, None if b is None else b.detach(), kind, rotated_pair=True, dtype=dtype,
        keep_z=True).z
    call = nv.gated_activation_backward if gated else nv.activation_backward
    back = call(dy, kept, kind, bias=bias, bias_type=F32)
    if bias:
        assert torch.equal(b.grad, back.dbias)
    dz = back.dz.to(BF16)
    q = linear._quantize("sr", dz, 3 * seed, 2 * seed + 1, ("row", "col"), "mx")
    wq = linear._quantize("sr", w.detach(), 3 * seed + 1, 2 * seed + 1, ("col",), "mx").col
    xq = linear._quantize("sr", x.detach(), 3 * seed + 2, 2 * seed + 1, ("col",), "mx").col
    for name, grad, operands in (("dx", x.grad, (q.row, wq)), ("dw", w.grad, (q.col, xq))):
        ref, tol = product(*operands)
        within(grad, ref, HALF[BF16] * (ref.abs() + tol) + 1.01 * tol, name)


def test_same_as_the_plain_layer():
    """Without an epilogue the layer is the FP32 one, rounded."""
    g = gen(1)
    x, dy = randn(g, 256, 128).to(BF16), randn(g, 256, 256).to(BF16)
    plain = QuartetLinear(128, 256, seed=3, scheme="sr", device=DEV, scales="mx")
    other = QuartetLinear(128, 256, seed=3, scheme="sr", device=DEV, scales="mx", dtype=BF16)
    other.load_state_dict(plain.state_dict())
    xs = [x.clone().requires_grad_() for _ in range(2)]
    ys = [m(t) for m, t in zip((plain, other), xs)]
    assert ys[0].dtype == F32 and ys[1].dtype == BF16
    assert torch.equal(ys[0].to(BF16), ys[1])
    for y in ys:
        y.backward(dy.to(y.dtype))
    assert torch.equal(xs[0].grad, xs[1].grad)
    assert torch.equal(plain.weight.grad, other.weight.grad)


def test_gradients_that_nobody_asks_for():
    g = gen(2)
    layer = QuartetLinear(128, 128, seed=1, scheme="sr", device=DEV, scales="mx", bias=True,
                          activation="gelu", dtype=BF16)
    x = randn(g, 128, 128).to(BF16)
    dy = randn(g, 128, 128).to(BF16)

    def grads(*wanted):
        layer._seed = 1
        t = x.clone().requires_grad_("x" in wanted)
        layer.weight.requires_grad_("w" in wanted)
        layer.bias.requires_grad_("b" in wanted)
        layer.weight.grad = layer.bias.grad = None
        layer(t).backward(dy)
        return dict(x=t.grad, w=layer.weight.grad, b=layer.bias.grad)
    full = grads("x", "w", "b")
    for wanted in ("x", "w", "b", "xb", "wb"):
        for name, t in grads(*wanted).items():
            assert (t is not None) == (name in wanted)
            assert t is None or torch.equal(t, full[name]), (wanted, name)
    with torch.no_grad():
        layer._seed = 1
        y = layer(x)
    assert not y.requires_grad


def test_no_second_derivatives():
    layer = QuartetLinear(128, 128, device=DEV, scheme="sr", scales="mx", activation="silu",
                          dtype=BF16)
    x = torch.randn(128, 128, device=DEV).to(BF16).requires_grad_()
    grad, = torch.autograd.grad(layer(x).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        grad.sum().backward()


def test_captured_step():
    """Forward, backward and update of a gated layer in one graph, replayed with other work between;
    each replay gives the eager step's bits."""
    def build():
        torch.manual_seed(0)
        up = QuartetLinear(128, 256, seed=7, scheme="sr", device=DEV, scales="mx", gated=True,
                           activation="silu", dtype=BF16)
        down = QuartetLinear(256, 128, seed=9, scheme="sr", device=DEV, scales="mx", dtype=BF16)
        return up, down, [up.weight, down.weight]
    g = gen(6)
    x, dy = randn(g, 128, 128).to(BF16), randn(g, 128, 128).to(BF16)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    hyper = dict(lr=1e-2, seed=3, max_norm=1.0)

    def run(up, down, params, states, step):
        up._seed, down._seed = 7, 9
        y = down(up(x), residual=x)
        grads = torch.autograd.grad(y, params, dy)
        nv.adamw_step(params, grads, states, step=step, norm=nv.grad_norm(grads), **hyper)
        return y
    up, down, params = build()
    states = [nv.adamw_state(p, 8, master=True) for p in params]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                 # what the first call allocates
        scratch = build()
        run(*scratch, [nv.adamw_state(p, 8, master=True) for p in scratch[2]], 1)
    torch.cuda.current_stream().wait_stream(side)
    del scratch
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step += 1
        y = run(up, down, params, states, step)
    eager = build()
    es = [nv.adamw_state(p, 8, master=True) for p in eager[2]]
    for k in range(1, 4):
        x.copy_(randn(g, 128, 128))
        graph.replay()
        torch.cuda.synchronize()
        ref = run(*eager, es, k).detach()
        assert torch.equal(y, ref)
        for p, q in zip(params, eager[2]):
            assert torch.equal(p, q)
        for s, t in zip(states, es):
            assert all(torch.equal(a, b) for a, b in zip(s, t))


def test_refusals():
    for kwargs in (dict(bias=True), dict(activation="gelu"), dict(gated=True), dict(dtype=BF16)):
        with pytest.raises(ValueError, match="scales=\"mx\""):
            QuartetLinear(128, 128, **kwargs)
    with pytest.raises(ValueError, match="unknown activation"):
        QuartetLinear(128, 128, scheme="sr", scales="mx", activation="tanh")
    x = torch.zeros(128, 128, device=DEV, dtype=BF16)
    layer = QuartetLinear(128, 128, device=DEV)
    with pytest.raises(ValueError, match="a residual needs"):
        layer(x, residual=x)
    gated = QuartetLinear(128, 128, scheme="sr", device=DEV, scales="mx", gated=True, dtype=BF16)
    with pytest.raises(ValueError, match="no residual"):
        gated(x, residual=x)
    with pytest.raises(ValueError, match="multiple of 128"):
        gated(x[:100])


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                        "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("bits", [32, 8])
def test_example_with_gated_blocks(bits):
    """The example's model with gated blocks and AdamW, run together for a few steps."""
    losses, norms = _example().train(steps=4, vocabulary=200, hidden=128, layers=2, tokens=256,
                                     feed_forward="gated", moments=bits)
    assert len(losses) == len(norms) == 4
    assert all(0 < t < 100 for t in losses) and all(0 < t < 1000 for t in norms)
