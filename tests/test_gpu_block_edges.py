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
