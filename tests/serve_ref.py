"""Plain implementations, in 64 bits on the CPU, of the serving operators: the paged cache, its
attention and draft verification.  Loops over requests, heads and tokens; no tensor of the
library's code is used."""
from __future__ import annotations

import math

import numpy as np
import torch

E4M3 = torch.float8_e4m3fn


def e4m3_table():
    """The 127 non-negative finite e4m3 values, in code order."""
    v = []
    for c in range(127):
        e, m = c >> 3, c & 7
        v.append(m * 2.0**-9 if e == 0 else (1 + m / 8) * 2.0**(e - 7))
    return np.array(v)


_TABLE = e4m3_table()


def quantise(x):
    """Rows of float64 [..., D] -> (codes uint8, scale bytes uint8) by the definition: s the
    smallest integer >= -100 (at most 119) with amax <= 448 * 2^s, codes the nearest e4m3 value
    (ties to the even code), saturating."""
    x = np.asarray(x, dtype=np.float64)
    amax = np.abs(x).max(-1)
    s = np.zeros(amax.shape, dtype=np.int64)
    for i in np.ndindex(*amax.shape):
        a = amax[i]
        if a > 0:
            e = -100
            while e < 119 and a > 448.0 * 2.0**e:
                e += 1
            s[i] = e
    y = np.abs(x) / 2.0**s[..., None]
    y = np.minimum(y, 448.0)
    hi = np.searchsorted(_TABLE, y).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = y - _TABLE[lo], _TABLE[hi] - y
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(y == _TABLE[hi], hi, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8), (s + 127).astype(np.uint8)


def dequantise(codes, scales):
    """uint8 codes [..., D] and scale bytes [...] -> float64 values."""
    v = np.where(codes & 128, -1.0, 1.0) * np.concatenate([_TABLE, [np.nan]])[codes & 127]
    out = v * 2.0**(scales.astype(np.float64) - 127)[..., None]
    out[scales == 255] = np.nan
    return out


def attention(q, k, v, n_kv, scale, causal=True, window=0):
    """One request: q [n, Hq, D], k, v [kv, H, D] float64 (token j of the cache).  Returns o, lse and
    the sum of p * |v| of every output (what roundings of p are measured against)."""
    n, Hq, D = q.shape
    H = k.shape[1]
    o, lse, mag = np.zeros((n, Hq, D)), np.full((n, Hq), -np.inf), np.zeros((n, Hq, D))
    for i in range(n):
        pos = n_kv - n + i
        hi = min(n_kv, pos + 1) if causal else n_kv
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            continue
        for h in range(Hq):
            g = h // (Hq // H)
            s = scale * (k[lo:hi, g] @ q[i, h])
            m = s.max()
            p = np.exp(s - m)
            lse[i, h] = m + math.log(p.sum())
            p /= p.sum()
            o[i, h] = p @ v[lo:hi, g]
            mag[i, h] = p @ np.abs(v[lo:hi, g])
    return o, lse, mag


def verify(target, draft, cu, ids, u, u_draw, max_draft):
    """Whole-number draft verification in Python integers; target, draft numpy float32."""
    B = len(cu) - 1
    out = np.full((B, max_draft + 1), -1, dtype=np.int64)
    length = np.zeros(B, dtype=np.int64)
    for b in range(B):
        first, n = cu[b], cu[b + 1] - cu[b]
        c = 0
        while c < n:
            x = ids[first + c]
            if not 0 <= x < target.shape[1]:
                break
            qx = float(draft[first + c, x]) if draft is not None else 1.0
            ux = min(max(float(u[first + c]), 0.0), 1 - 2.0**-24)
            if not ux * qx < float(target[first + b + c, x]):
                break
            out[b, c] = x
            c += 1
        p = target[first + b + c].astype(np.float32)
        r = p
        if c < n:
            q = draft[first + c] if draft is not None else np.zeros_like(p)
            if draft is None and 0 <= ids[first + c] < len(p):
                q[ids[first + c]] = 1.0
            r = p - q

        def weights(r):
            r = np.where(np.isnan(r), 0, r).clip(0, 1).astype(np.float64)
            return np.floor(r * 2.0**40).astype(np.int64)

        w = weights(r)
        if w.sum() == 0:
            w = weights(p)
        total = int(w.sum())
        if total:
            m = int(math.floor(min(max(float(u_draw[b]), 0.0), 1 - 2.0**-24) * 2**24))
            want = m * total >> 24
            out[b, c] = int(np.searchsorted(np.cumsum(w), want, side="right"))
        length[b] = c + 1
    return out, length
