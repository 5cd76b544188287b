"""A small language model trained for a few steps with this package's operators together: layer
norm, NVFP4 linear layers (MS-EDEN backward), the linear head's cross entropy without logits,
and gradient clipping before the update.

    python examples/train_step.py --steps 60
    python examples/train_step.py --steps 60 --feed-forward gated --moments 8

The second line's blocks are gated and run on the MXFP4 recipe, with activation, gating and residual in
the products' kernels, and its update is this package's AdamW, which clips on the way.

Data is synthetic: each token follows from the one before by a fixed permutation of the vocabulary,
one in ten is replaced by a random one, and a tenth of the positions do not count (prompts).
"""
import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import unbiased_nvfp4_gradient_amd as nv  # noqa: E402
from unbiased_nvfp4_gradient_amd.linear import QuartetLinear  # noqa: E402

IGNORE = -100


class Block(torch.nn.Module):
    """x + down(gelu(up(layer norm of x)))."""

    def __init__(self, hidden, seed, device):
        super().__init__()
        self.norm = nv.LayerNorm(hidden, device=device)
        self.up = QuartetLinear(hidden, 4 * hidden, seed=seed, device=device)
        self.down = QuartetLinear(4 * hidden, hidden, seed=seed + 1000, device=device)

    def forward(self, x):
        a = F.gelu(self.up(self.norm(x))).to(torch.bfloat16)
        return x + self.down(a).to(torch.bfloat16)


class GatedBlock(torch.nn.Module):
    """x + down(silu(gate) up) of the layer norm of x, on the MXFP4 recipe."""

    def __init__(self, hidden, seed, device):
        super().__init__()
        mx = dict(scheme="sr", device=device, scales="mx", dtype=torch.bfloat16)
        self.norm = nv.LayerNorm(hidden, device=device)
        self.up = QuartetLinear(hidden, 4 * hidden, seed=seed, gated=True, activation="silu", **mx)
        self.down = QuartetLinear(4 * hidden, hidden, seed=seed + 1000, bias=True, **mx)

    def forward(self, x):
        return self.down(self.up(self.norm(x)), residual=x)


class Model(torch.nn.Module):
    def __init__(self, vocabulary, hidden, layers, device, block=Block):
        super().__init__()
        self.embedding = torch.nn.Embedding(vocabulary, hidden, device=device,
                                            dtype=torch.bfloat16)
        self.blocks = torch.nn.ModuleList(block(hidden, 10 * k, device) for k in range(layers))
        self.norm = nv.LayerNorm(hidden, device=device)
        self.head = torch.nn.Parameter(torch.empty((vocabulary, hidden), device=device,
                                                   dtype=torch.bfloat16))
        torch.nn.init.normal_(self.head, std=hidden ** -0.5)

    def forward(self, tokens, target):
        x = self.embedding(tokens)
        for block in self.blocks:
            x = block(x)
        return nv.linear_cross_entropy(self.norm(x), self.head, target, ignore_index=IGNORE)


def batches(vocabulary, tokens, device, seed):
    """(tokens, targets) without end."""
    g = torch.Generator(device=device).manual_seed(seed)
    follows = torch.randperm(vocabulary, generator=g, device=device)
    while True:
        x = torch.randint(vocabulary, (tokens,), generator=g, device=device)
        y = follows[x]
        noise = torch.rand((tokens,), generator=g, device=device)
        y = torch.where(noise < 0.1, x.flip(0), y)
        yield x, torch.where(noise > 0.9, torch.full_like(y, IGNORE), y)


def train(steps, vocabulary=500, hidden=256, layers=2, tokens=2048, rate=2e-2, max_norm=0.25,
          seed=0, device="cuda:0", report=None, feed_forward="gelu", moments=None):
    """(losses, gradient norms before clipping) of a training run with Adam or, where `moments` gives
    the bits of its moments, this package's AdamW with float32 masters."""
    torch.manual_seed(seed)
    model = Model(vocabulary, hidden, layers, device,
                  GatedBlock if feed_forward == "gated" else Block)
    params = list(model.parameters())
    if moments:
        optimizer = nv.AdamW(params, lr=rate, bits=moments, master=True, seed=seed)
    else:
        optimizer = torch.optim.Adam(params, lr=rate)
    losses, norms = [], []
    for step, (x, y) in zip(range(steps), batches(vocabulary, tokens, device, seed)):
        optimizer.zero_grad(set_to_none=True)
        loss = model(x, y)
        loss.backward()
        grads = [p.grad for p in params]
        if moments:
            norms.append(nv.grad_norm(grads))
            optimizer.step(norm=norms[-1], max_norm=max_norm)
        else:
            norms.append(nv.clip_grads(grads, max_norm))
            optimizer.step()
        losses.append(loss.detach())
        if report and step % report == 0:
            print(f"step {step:4d}  loss {float(losses[-1]):.4f}  "
                  f"gradient norm {float(norms[-1]):.4f}", flush=True)
    return torch.cat(losses).tolist(), torch.cat(norms).tolist()


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--vocabulary", type=int, default=500)
    ap.add_argument("--hidden", type=int, default=256, help="a multiple of 128")
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--tokens", type=int, default=2048, help="a multiple of 128")
    ap.add_argument("--feed-forward", choices=("gelu", "gated"), default="gelu")
    ap.add_argument("--moments", type=int, choices=(32, 8), help="bits of AdamW's moments")
    args = ap.parse_args()
    losses, _ = train(args.steps, args.vocabulary, args.hidden, args.layers, args.tokens, report=10,
                      feed_forward=args.feed_forward, moments=args.moments)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f} (uniform guess "
          f"{math.log(args.vocabulary):.4f})")


if __name__ == "__main__":
    main()
