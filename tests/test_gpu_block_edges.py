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
