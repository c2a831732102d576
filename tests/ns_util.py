"""Newton-Schulz steps in 64 bits and in plain fp32, and the error bound of their tests.

A product of two fp16 terms per operand drops at most 2^-22 of each product where fp32 rounds
2^-24: errors are held to four times those of the same steps with fp32 products, and, where these
happen to vanish, to one unit of 2^-22 for each of a run's 15 products and its first operand, 16 in
all, in the 2-norm of the result.  The result is rounded once to its type.

The low terms end at 2^-24 of operands scaled to 2^15 at most: X is held to half of that, 2^-40 an
element, whatever its size, 2^-40 sqrt(rows cols) in norm, which the steps multiply by up to their
first coefficients.  With a norm of at least eps this is far below the rest; a matrix whose
norm is far below eps, and X with it, is held to this alone."""
import torch

import linear_util as lu

COEFFS = (3.4445, -4.7750, 2.0315)


def steps_in(g, dtype, steps=5, coeffs=None, eps=1e-7):
    x = g.to(dtype)
    x = x / x.square().sum().sqrt().clamp(min=eps)
    tall = x.shape[0] > x.shape[1]
    if tall:
        x = x.t().contiguous()
    for k in range(steps):
        a, b, c = (float(torch.tensor(v, dtype=torch.float32)) for v in (COEFFS if coeffs is None else coeffs[k]))   # as the call takes them
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if tall else x


def check(got, g, what="result", **k):
    want, plain = steps_in(g, torch.float64, **k), steps_in(g, torch.float32, **k)
    size = float(want.norm())
    err = float((got.double() - want).norm())
    gain = 1.0
    for a, _, _ in k.get("coeffs") or [COEFFS] * k.get("steps", 5):
        gain *= max(1.0, abs(a))
    held = gain * 2.0 ** -40 * (want.shape[0] * want.shape[1]) ** 0.5
    tol = 4 * float((plain.double() - want).norm()) + 16 * 2.0 ** -22 * size + lu.OUT_ULP[got.dtype] * size + held
    assert err <= tol, f"{what}: {err / (size or 1):.3g} of the norm off, {err / tol:.3g} of the bound"
    return err / (size or 1.0)


def gradient(rows, cols, gen, rank=4, dtype=torch.float32, std=1e-3):
    """Noise and as much again in a few strong directions."""
    u, v = (torch.randn(n, rank, generator=gen, device="cuda") for n in (rows, cols))
    return ((torch.randn(rows, cols, generator=gen, device="cuda") + 0.5 * (u @ v.t())) * std).to(dtype)
