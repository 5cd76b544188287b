"""Layer norm, the linear head's cross entropy and clipping at the ends of their ranges, against
plain 64-bit implementations.  Tolerances count roundings, as in test_gpu_training.py: U is half a
step of float32, HALF[t] half a step of type t."""
import pytest
import torch

import unbiased_nvfp4_gradient_amd as nv
from test_gpu_training import BF16, DEV, F16, U, within

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
