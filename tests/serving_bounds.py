"""An error bound for attention outputs that does not grow with the length where
nothing is lost.

Let u = finfo.eps / 2 (half a step of the 16-bit type relative to the value)
and ds as in the serving tests: how far a score can be off. A softmax numerator
is off by a factor within e^(+-ds) (1 + 2^-21), the denominator too: dp
together. Numerators are taken relative to a running maximum, which is never
above the row's own maximum, so the largest is at least 1 and so is the
denominator; where partial sums are joined, each is scaled by at most 1.
Rounding a numerator to 16 bits costs u of it, or, below fp16's smallest normal
2^-14, half of 2^-24: over the row at most 2^-25 sum |v|, divided by a
denominator of at least 1. The output's rounding costs u of its value (2^-25
below 2^-14).
"""
import numpy as np
import torch

D = 128


def score_error(size):
    """`size`: scale * sum |q||k|. D roundings of an fp32 sum that may truncate, and the scale's."""
    return size * (2 * D * 2.0 ** -24 + 2.0 ** -22)


def o_bound(ref, pv, size, dtype, sum_v):
    """ref, pv = sum p|v|, sum_v = sum |v| over the attended keys: [.., D]; size [..]."""
    u = torch.finfo(dtype).eps / 2
    dp = 2 * np.expm1(np.asarray(score_error(size))) + 2.0 ** -19
    tol = (dp[..., None] + u) * pv * (1 + u) + u * np.abs(ref) + 1e-30
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25 * (1 + 2.0 ** -9) * sum_v + 2.0 ** -25
    return tol


def check(got, ref, pv, size, dtype, sum_v, what):
    tol = o_bound(ref, pv, size, dtype, sum_v)
    err = np.abs(got - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size}, worst {np.nanmax(err / tol):.2f} of the bound"
