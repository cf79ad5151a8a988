"""Error bounds of the FFN operators, from their arithmetic.

fp32 tensor-core sums of FP8 products: the products are exact; each
instruction adds 32 of them to the accumulator.  Allowed per instruction: one
fp32 step (2^-23, truncation included) of the sum of absolute terms, twice (the
sum inside the instruction and the addition to the accumulator); plus the
additions that join split sums, at most 16 of half a step each.  Hence
    |error of a sum| <= (2 K / 32 + 16) * 2^-23 * (sum of absolute terms).
The scales, bias, residual and weighted sums are single fp32 operations: half a
step (2^-24) each of values no larger than the ones added here, 2^-20 in all.
Activations: |derivative| <= 1.13 (GELU's maximum 1.129; SiLU's 1.1), and an own
relative error of at most 2^-17 (the GELU fit's 3.6e-6 with the intrinsics' error
of 2^-21; e^-z multiplies a rounding of z, |z| * 2^-24, at most 2^-17 for |z| < 90).
fp16 output: half a step, 2^-11 of the value, or 2^-25 below the normal range.
"""
import numpy as np

F16_HALF = 2.0 ** -11
F16_TINY = 2.0 ** -25
ACT_SLOPE = 1.13
ACT_REL = 2.0 ** -17
ONE_OPS = 2.0 ** -20


def sum_bound(K, terms):
    return (2.0 * ((K + 31) // 32) + 16.0) * 2.0 ** -23 * terms


def round_f16(bound, value):
    """Bound after rounding to fp16: half a step of the largest value the unrounded one may have."""
    return bound + np.maximum(F16_HALF * (np.abs(value) + bound), F16_TINY)


def assert_within(got, ref, bound, what=""):
    got = np.asarray(got, dtype=np.float64)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~(np.abs(got - ref) <= bound)   # NaN counts as bad
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} outside the bound; first at {i}: "
                             f"got {got[i]!r}, exact {ref[i]!r}, bound {np.broadcast_to(bound, ref.shape)[i]!r}")


def linear_epilogue_bound(K, y, terms, residual=None):
    """y: unrounded result; terms: absolute product terms."""
    a = np.abs(y) + (np.abs(np.asarray(residual, dtype=np.float64)) if residual is not None else 0.0)
    b = ACT_SLOPE * (sum_bound(K, terms) + ONE_OPS * terms) + (ACT_REL + ONE_OPS) * 2.0 * a
    return round_f16(b, y)


def moe_hidden_bound(K, h, z, terms, gated):
    """Bound of the fp16 hidden rows."""
    F = h.shape[1]
    e = sum_bound(K, terms) + ONE_OPS * terms
    if not gated:
        return round_f16(ACT_SLOPE * e + (ACT_REL + ONE_OPS) * np.abs(h), h)
    # act(a) * b: |act(a)| <= |a|
    ea = ACT_SLOPE * e[:, :F] + ACT_REL * np.abs(z[:, :F])
    return round_f16(ea * (np.abs(z[:, F:]) + e[:, F:]) + np.abs(z[:, :F]) * e[:, F:] + ONE_OPS * np.abs(h), h)


def moe_out_bound(F, out, terms, residual=None):
    r = np.abs(np.asarray(residual, dtype=np.float64)) if residual is not None else 0.0
    return round_f16(sum_bound(F, terms) + ONE_OPS * (terms + np.abs(out) + r), out)
