"""Inputs of attention whose scores are exact in fp32, whatever the order of their sums: whole numbers times a power of
two.  A softmax of any sharpness can then be held to the roundings of its probabilities and of its output alone, where
latent_ref's bound for real numbers (every product's rounding at its worst) lets anything pass."""
from __future__ import annotations

import numpy as np

import latent_ref as R


def whole(rng, *shape, most):
    return rng.integers(-most, most + 1, size=shape).astype(np.float64)


def growing(keys, steps, order="up"):
    """keys [kv, D] times 1 .. steps, in runs of the same factor: maxima that rise from run to run (order "up"), fall, or
    rise and fall."""
    kv = keys.shape[0]
    f = np.arange(kv) * steps // max(kv, 1) + 1
    if order == "down":
        f = f[::-1]
    elif order == "both":
        f = np.minimum(f, f[::-1]) * 2 - 1
    return keys * f[:, None]


def attention(q, k, v, seen, scale):
    """latent_ref.attention with the bound of a score's error for these inputs.  The kernels hold scores as powers of two: the
    factor scale * log2(e) is off by half a step (2^-24), the difference from the running maximum is rounded once
    (2^-24 of it), and so is what the accumulators are multiplied by when the maximum moves, a few times a row,
    each time of differences that sum to no more than the scores' range: 2^-21 of the largest score in all."""
    assert np.all(q == np.round(q)) and np.all(k == np.round(k)) and np.log2(scale) == np.round(np.log2(scale))
    largest = np.einsum("nhd,kd->nhk", np.abs(q), np.abs(k), optimize=True).max(initial=0)
    assert largest < 2**24  # every partial sum is a whole number of fp32's
    o, lse, mag, _ = R.attention(q, k, v, seen, scale)
    s = np.einsum("nhd,kd->nhk", q, k, optimize=True) * scale
    return o, lse, mag, np.full(lse.shape, np.abs(s).max(initial=0) * 2.0**-21)


def check(got_o, got_lse, ref, what):
    assert ref[3].max(initial=0) < 0.05, f"{what}: a bound that says nothing"
    R.check(got_o, got_lse, ref, what)


# q's and k's largest whole numbers, the power of two that scales their products, the keys' factors and their order
LATENT = {"flat": (2, 3, 2.0**-9, 1, "up"), "soft": (2, 3, 2.0**-5, 1, "up"), "sharp": (2, 3, 2.0**-2, 1, "up"),
          "one key": (2, 3, 1.0, 1, "up"), "rising": (2, 3, 2.0**-4, 20, "up"), "falling": (2, 3, 2.0**-4, 20, "down"),
          "rise and fall": (2, 3, 2.0**-4, 20, "both"), "rising far": (2, 3, 2.0**-1, 20, "up")}


def latent_numbers(rng, kind, n, heads, kv, width=576, values=512):
    """(q [n, heads, width], keys [kv, width], values, scale)."""
    a, b, scale, steps, order = LATENT[kind]
    keys = growing(whole(rng, kv, width, most=b), steps, order)
    return whole(rng, n, heads, width, most=a), keys, keys[:, :values], scale
