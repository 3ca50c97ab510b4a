"""Plain implementations, in 64 bits on the CPU, of latent attention (both forms), trees of drafted tokens and
the norms around a block.  Loops over requests; no code of the library's is used."""
from __future__ import annotations

import numpy as np

U_BF16 = 2.0**-8   # half a step of bf16, relative to the value
U_F32 = 2.0**-24


def rms(x, w, eps):
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w


def block_norm(y, pre, resid=None, post=None, gate=None, scale=1.0, eps=1e-6):
    x = y if post is None else rms(y, post, eps)
    if gate is not None:
        x = x * gate
    r = scale * x + (0 if resid is None else resid)
    return r, None if pre is None else rms(r, pre, eps)


def chain(n, kv, causal=True, window=0):
    """Which of kv cached tokens each of a request's n newest sees, bool [n][kv]."""
    pos, j = np.arange(kv - n, kv)[:, None], np.arange(kv)[None]
    seen = np.ones((n, kv), dtype=bool)
    if causal:
        seen &= j <= pos
    if window:
        seen &= j > pos - window
    return seen


def branches(bits, n, kv):
    """The same for a tree: bits [n], bit j of a token's for the request's new token j."""
    seen = np.zeros((n, kv), dtype=bool)
    for i in range(n):
        for x in range(kv):
            j = x - (kv - n)
            seen[i, x] = j < 0 or j == i or bool(int(bits[i]) >> j & 1)
    return seen


def random_tree(rng, n):
    """Bits of a random tree's nodes, uint64 [n]: each node's ancestors and itself."""
    out = []
    for i in range(n):
        parent = int(rng.integers(-1, i)) if i else -1
        out.append((out[parent] if parent >= 0 else 0) | 1 << i)
    return np.array(out, dtype=np.uint64)


def attention(q, k, v, seen, scale):
    """One request, one key head: q [n, H, D], k [kv, D], v [kv, Dv], seen [n, kv].  Returns o, lse, the sum of
    p * |v| of every output (what roundings of p are measured against) and a bound of a score's error when its
    products are summed in fp32: D roundings of half a step of the sum of magnitudes, twice for sums that
    are cut instead of rounded."""
    n, H, D = q.shape
    s = np.einsum("nhd,kd->nhk", q, k, optimize=True) * scale
    s = np.where(seen[:, None], s, -np.inf)
    mag_s = np.einsum("nhd,kd->nhk", np.abs(q), np.abs(k), optimize=True) * scale
    err = (np.where(seen[:, None], mag_s, 0).max(-1, initial=0)) * D * 2 * U_F32
    m = s.max(-1, initial=-np.inf)
    p = np.exp(s - np.where(np.isneginf(m), 0, m)[..., None])
    total = p.sum(-1)
    with np.errstate(divide="ignore"):
        lse = m + np.log(total)
    p /= np.where(total == 0, 1, total)[..., None]
    return (np.einsum("nhk,kd->nhd", p, v, optimize=True), lse, np.einsum("nhk,kd->nhd", p, np.abs(v), optimize=True),
            err)


def check(got_o, got_lse, ref, what):
    """|o - exact| <= half a step of bf16 of o (its rounding) + half a step of every probability's part + what a
    score's error does to the probabilities (e^err - 1 of them, up and down: twice) + 2^-20 of them for the exponential,
    the sum and the division.  lse: the score's error and 2^-20 of itself, and of 1 for the logarithm near 0."""
    o, lse, mag, err = ref
    empty = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got_lse), empty), f"{what}: rows that see nothing"
    assert np.all(got_o[empty] == 0), f"{what}: rows that see nothing"
    bound = U_BF16 * np.abs(o) + (U_BF16 * (1 + 2.0**-6) + 2 * np.expm1(err)[..., None] + 2.0**-20) * mag + 1e-30
    bad = ~(np.abs(got_o - o) <= bound)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outputs off, first {np.argwhere(bad)[:3].tolist()}"
    off = np.abs(got_lse - np.where(empty, 0, lse))[~empty]
    assert np.all(off <= (err + 2.0**-20 * (1 + np.abs(np.where(empty, 0, lse))))[~empty]), f"{what}: lse, {off.max()}"
