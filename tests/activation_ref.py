"""The activations in 64 bits, with bounds of what the kernels' FP32 forms may be off by, for the tests
of activations and of products with them."""
import math

import torch

U = 2.0 ** -24          # half a step of float32


def within(got, ref, tol, what):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), \
        f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err - tol).max())} " \
        f"above its bound (largest error {float(err.max())})"


def exact(z, kind):
    """(value, slope, bounds of both) in 64 bits, first order in U and 2% for the rest.  An
    exponential 2^x of the hardware and a reciprocal are off by 2 U (one unit in the last place); an
    exponential's argument off by r relative makes it off by |argument| r (natural logarithm)."""
    z = z.double()
    if kind in ("none", "relu"):
        on = z > 0 if kind == "relu" else torch.ones_like(z, dtype=torch.bool)
        zero = torch.zeros_like(z)
        return torch.where(on, z, zero), on.double(), zero, zero
    if kind == "gelu":
        low = 0.5 * torch.erfc(-z / math.sqrt(2))
        up = 0.5 * torch.erfc(z.abs() / math.sqrt(2))          # |z|'s upper part
        phi = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        slope = low + z * phi
        # density: three roundings of its argument z^2 / 2 (log2 e, two products), 2 U of its own.
        # upper part P(t) density, t = 1 / (1 + 0.304 |z|): the fit 1.6 U; Horner's rule, whose partial
        # sums at t = 1 (worst) add to 3.1 times their last; t, off by 3 U (sum and reciprocal), times
        # t P'(t) / P(t) <= 2.63; two products
        density = (1.5 * z * z + 2) * U
        rel = (1.6 + 3.1 + 3 * 2.63 + 2) * U + density
        part = rel * up + U * (z >= 0) * low                     # of the lower part
        value_tol = z.abs() * part + U * (z * low).abs()
        # z / sqrt(2 pi): the constant and a product; the sum's own rounding
        slope_tol = part + z.abs() * phi * (density + 2 * U) + U * slope.abs()
        return z * low, slope, 1.02 * value_tol + 1e-35, 1.02 * slope_tol + 1e-35
    if kind == "silu":
        x, du, r = z, torch.ones_like(z), 2 * U                 # log2 e and its product
        rest = U
    else:
        # x = 2 sqrt(2 / pi) (z + 0.044715 z^3): 3 U of the cubic term, the sum, the constant and its
        # product make 6 U, then log2 e and its product; x' = constants, product and sum 4 U
        k = 2 * math.sqrt(2 / math.pi)
        x, du, r = k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z), 8 * U
        rest = 6 * U                                            # of 1 - s, its product with z, and x'
    s, q = torch.sigmoid(x), torch.sigmoid(-x)
    rel = q * (x.abs() * r + 2 * U) + 3 * U                     # e^-x enters s by 1 - s; sum, reciprocal
    slope = s * (1 + z * q * du)
    # 1 - s is off by s's error; the sum with 1, the product with s
    slope_tol = (rel + 2 * U) * slope.abs() + s * z.abs() * du * (s * rel + q * rest)
    # where e^-x is infinite, s is below 2^-128
    return z * s, slope, 1.02 * (rel + U) * (z * s).abs() + 1e-35, 1.02 * slope_tol + 1e-35
