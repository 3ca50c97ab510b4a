"""Attention over an e4m3 cache whose scales lie far apart: a row's output goes by the keys that it sees
and by their weights, not by the largest scale that stands beside them."""
import math

import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from serve_ref import E4M3, attention
from test_gpu_attn import DEV, Case

pytestmark = pytest.mark.gpu
K, V = 0, 1


class Ranges(Case):
    """A Case on an e4m3 cache with scale bytes (and codes) of one's own."""

    def __init__(self, *a, **kw):
        self.page = kw.get("page", 16)
        super().__init__(*a, dtype="e4m3", **kw)

    def at(self, b, j):
        return int(self.host_table[b, j // self.page]), j % self.page

    def set_bytes(self, what, byte):
        """byte(b, j) -> the scale byte of token j of request b for key (what = K) or value rows, or None."""
        self.host_table = self.table.cpu()
        keep = self.keep.cpu()
        for b, kv in enumerate(self.kv_lens):
            for j in range(kv):
                to = byte(b, j)
                if to is not None:
                    page, at = self.at(b, j)
                    old = keep[what, page, :, at].numpy().astype(np.float64)
                    (self.k, self.v)[what][b][j] *= 2.0**(to - old)[:, None]
                    keep[what, page, :, at] = torch.as_tensor(to)
        self.keep.copy_(keep)

    def set_codes(self, what, code):
        """code(b, j) -> values of token j's row before its scale (e4m3 numbers, broadcast to [heads][head_dim]), or None."""
        self.host_table = self.table.cpu()
        pool, keep = self.pool.view(torch.uint8).cpu(), self.keep.cpu()
        for b, kv in enumerate(self.kv_lens):
            for j in range(kv):
                to = code(b, j)
                if to is not None:
                    page, at = self.at(b, j)
                    x = torch.as_tensor(to, dtype=torch.float32).expand(self.H, self.D).contiguous().to(E4M3)
                    pool[what, page, :, at] = x.view(torch.uint8)
                    s = keep[what, page, :, at].numpy().astype(np.float64)
                    (self.k, self.v)[what][b][j] = x.double().numpy() * 2.0**(s - 127)[:, None]
        self.pool.view(torch.uint8).copy_(pool)

    def set_q(self, q):
        self.q = q.to(torch.bfloat16)
        self.qd[:, :self.Hq] = self.q.to(DEV)

    def check_o(self, skip=None, **kw):
        """The bound of Case.check, down to bf16's subnormals (2^-133).  skip: a row of every request that is not asked for."""
        o, lse = self.run(**kw)
        assert int(self.err.item()) == 0
        first = 0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            q = self.q[first:first + n].double().numpy()
            ro, rl, mag = attention(q, self.k[b], self.v[b], kv, self.scale, self.causal, self.window)
            go, gl = o[first:first + n], lse[first:first + n]
            if skip is not None:
                go[skip], gl[skip] = ro[skip], rl[skip]
            bad = ~(np.abs(go - ro) <= 2.0**-8 * np.abs(ro) + (2.0**-8 + 2.0**-12) * mag + 2.0**-133)
            assert not bad.any(), f"request {b} (n {n}, kv {kv}): {bad.sum()} of {bad.size} outputs off, first " \
                                  f"{np.argwhere(bad)[:3].tolist()}: {go[bad][:3]} for {ro[bad][:3]}"
            assert np.abs(gl - rl).max() <= 1.2e-4, f"request {b}: lse"
            first += n


# rows a head: 4 * n.  Up to 32 are one kernel's, more another's.
@pytest.mark.parametrize("n", [2, 8, 20, 150])
@pytest.mark.parametrize("what", [K, V])
@pytest.mark.parametrize("gap", [12, 25, 40, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_scales_of_tokens_that_a_row_does_not_see(n, what, gap, D):
    """The last token's key or value is 2^gap larger, and only the last row sees it.  (That row's scores go past
    what fp32 tells apart where it is the key: not asked for.)"""
    c = Ranges([n, n], [n, n], D=D, seed=n)
    c.set_bytes(what, lambda b, j: (120 if what == K else 100) + (gap if j == n - 1 else 0))
    c.check_o(skip=n - 1 if what == K else None)
    c = Ranges([n], [n + 3], D=D, window=4, seed=n)  # the first one's, which the window leaves to the first row
    c.set_bytes(what, lambda b, j: (120 if what == K else 100) + (gap if j == 0 else 0))
    c.check_o(skip=0 if what == K else None)


@pytest.mark.parametrize("n", [1, 6, 70])
@pytest.mark.parametrize("weight", [0, 1, 2])
@pytest.mark.parametrize("gap", [22, 30, 60, 100])
def test_large_values_of_little_weight(n, weight, gap):
    """One value 2^gap larger than the rest, whose key takes it to a weight of about 2^-13, 2^-26 or 2^-52: what
    it adds counts beside the rest, or not at all, and the rest keeps its precision."""
    for place in (0, 130, 256, 620):
        c = Ranges([n, n], [700, 257], seed=gap + place)
        c.set_q(c.q.float().abs())
        c.set_bytes(V, lambda b, j: 118 + j % 4)
        c.set_codes(K, lambda b, j: -256.0 if j == place else None)
        c.set_bytes(K, lambda b, j: 119 + weight if j == place else None)
        c.set_bytes(V, lambda b, j: 118 + gap if j == place else None)
        c.check_o()


@pytest.mark.parametrize("n", [1, 6, 70])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_ctas", [0, 3])
def test_random_scales(n, D, max_ctas):
    """Every value row its own scale in moe_kv_write's whole range; keys from ordinary ones down to 2^-60."""
    rng = np.random.default_rng(n)
    c = Ranges([n, n, n], [300, 75, 900], D=D, page=32)
    c.set_bytes(V, lambda b, j: rng.integers(27, 247, size=c.H))
    c.check_o(max_ctas=max_ctas)
    c = Ranges([n, n, n], [300, 75, 900], D=D, page=32)
    c.set_bytes(K, lambda b, j: rng.integers(60, 121, size=c.H))
    c.check_o(max_ctas=max_ctas)


@pytest.mark.parametrize("n", [1, 6, 70])
@pytest.mark.parametrize("bytes_", [(60, 120, 180, 100), (180, 100, 60, 130), (110, 128, 118, 122), (40, 41, 240, 42)])
@pytest.mark.parametrize("max_ctas", [0, 1])
def test_columns_that_only_some_tokens_fill(n, bytes_, max_ctas):
    """Four stretches of tokens with scales of their own, each with values in a quarter of the columns: a
    column has no part of the larger ones, so it has to come out as if they were not there.  (Stretches
    up to 2^200 apart in one request: a column 2^-120 and more below another may be lost, so the
    smallest of the last set is not asked for.)"""
    D = 128
    c = Ranges([n, n], [820, 300], D=D, page=64)

    def part(b, j):
        return min(j * 4 // c.kv_lens[b], 3)

    c.set_bytes(V, lambda b, j: bytes_[part(b, j)])
    rng = np.random.default_rng(0)

    def code(b, j):
        x = np.zeros((c.H, D), np.float32)
        x[:, part(b, j) * 32:part(b, j) * 32 + 32] = rng.uniform(1, 400, size=(c.H, 32))
        return x

    c.set_codes(V, code)
    if max(bytes_) - min(bytes_) > 150:
        cols = [i for i in range(4) if max(bytes_) - bytes_[i] <= 110]
        run = c.run

        def only(**kw):
            o, lse = run(**kw)
            first = 0
            for b, m in enumerate(c.q_lens):
                q = c.q[first:first + m].double().numpy()
                ro = attention(q, c.k[b], c.v[b], c.kv_lens[b], c.scale)[0]
                for i in range(4):
                    if i not in cols:  # within 2^-110 of the largest
                        s = slice(i * 32, i * 32 + 32)
                        assert (np.abs(o[first:first + m, :, s] - ro[..., s]) <= 2.0**(max(bytes_) - 127 - 110)).all()
                        o[first:first + m, :, s] = ro[..., s]
                first += m
            return o, lse

        c.run = only
    c.check_o(max_ctas=max_ctas)


@pytest.mark.parametrize("n", [1, 6, 70])
def test_the_smallest_scales(n):
    """A scale byte b stands for 2^(b - 127) down to b = 0; values of 2^-127 to 2^-111 come out as such."""
    c = Ranges([n, n], [200, 90])
    c.set_bytes(V, lambda b, j: j % 8)
    c.check_o()
    c.set_bytes(V, lambda b, j: 0)
    c.check_o()
    c = Ranges([n, n], [200, 90])
    c.set_q(c.q.float() * 2.0**100)  # scores of about 2^-13 from keys of about 2^-113
    c.set_bytes(K, lambda b, j: j % 4)
    c.check_o()


@pytest.mark.parametrize("n", [1, 6, 70])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_scale_near_the_smallest(n, dtype):
    """All scores 0 or next to it: the masked ones must not become -inf * 0."""
    for scale in (2.0**-60, 2.0**-126):
        c = Case([n, n], [200, 90], dtype=dtype, scale=scale)
        c.q = c.q * 0
        c.qd.zero_()
        c.check()


@pytest.mark.parametrize("n", [1, 70])
def test_weights_of_a_long_context(n):
    """One key with the weight of all the others together, each of which has 2^-14 of it: they add up."""
    kv = 16385
    c = Ranges([n], [kv], Hq=2, H=1, page=64)
    c.set_q(torch.ones_like(c.q))
    s = 14 * math.log(2) / c.scale / 128  # of each of 128 columns
    c.scale *= s
    c.args = c.make_args()
    c.set_codes(K, lambda b, j: 256.0 if j == 5 else 0.0)
    c.set_bytes(K, lambda b, j: 119)
    c.set_codes(V, lambda b, j: 0.0 if j == 5 else None)
    c.set_bytes(V, lambda b, j: 120)
    c.check_o()
