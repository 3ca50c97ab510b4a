"""Latent attention (expanded form) on the GPU against a plain implementation in 64 bits."""
import numpy as np
import pytest
import torch

from latent_ref import attention, chain, check
from moe_expert_dispatch_route_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """Rows of keys and values that belong to no request are NaN."""

    def __init__(self, q_lens, kv_lens, heads=2, causal=True, seed=0, std=1.0, scale=192**-0.5, pad=0):
        rng = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.heads, self.causal, self.scale = q_lens, kv_lens, heads, causal, scale
        T, S = sum(q_lens), sum(kv_lens)
        rand = lambda *s: torch.tensor(rng.standard_normal(s) * std).to(torch.bfloat16)
        self.q, self.k, self.r, self.v = rand(T, heads, 192), rand(S, heads, 128), rand(S, 64), rand(S, heads, 128)
        nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=DEV)
        self.qd = nan(T + 3, heads, 192 + 8 * pad)
        self.kv = nan(S + 5, heads + pad, 256)  # keys and values of a head side by side
        self.rd = nan(S + 5, 64 + 8 * pad)
        self.qd[:T, :, :192] = self.q.to(DEV)
        self.kv[:S, :heads, :128], self.kv[:S, :heads, 128:] = self.k.to(DEV), self.v.to(DEV)
        self.rd[:S, :64] = self.r.to(DEV)
        self.od = torch.full((T + 3, heads + pad, 128 + 8 * pad), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((T + 3, heads), 77.0, device=DEV)
        self.cu = torch.tensor([0] + np.cumsum(q_lens).tolist(), dtype=torch.int32, device=DEV)
        self.cu_kv = torch.tensor([0] + np.cumsum(kv_lens).tolist(), dtype=torch.int32, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.zeros(B.moe_attn_expanded_workspace_size(heads), dtype=torch.uint8, device=DEV)
        self.args = self.make_args()

    def make_args(self, max_q=None, max_kv=None, lse=True):
        h = self.heads
        return B.attn_expanded_args(self.qd[:, :, :192], self.kv[:, :h, :128], self.rd[:, :64], self.kv[:, :h, 128:],
                                    self.od[:, :h, :128], self.cu, self.cu_kv, max_q or max(self.q_lens),
                                    max_kv or max(self.kv_lens), self.scale, causal=self.causal,
                                    lse=self.lse if lse else None, workspace=self.ws, err_flag=self.err)

    def run(self, **kw):
        self.od.fill_(77.0)
        self.lse.fill_(77.0)
        B.moe_attn_expanded(self.args, **kw)
        torch.cuda.synchronize()
        T = sum(self.q_lens)
        return self.od[:T, :self.heads, :128].double().cpu().numpy(), self.lse[:T].double().cpu().numpy()

    def check(self, **kw):
        o, lse = self.run(**kw)
        assert int(self.err.item()) == 0
        assert int(self.ws[:4096].count_nonzero().item()) == 0, "the counters are left zero"
        a = e = 0
        d = lambda t: t.double().numpy()
        for b, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            for h in range(self.heads):
                k = np.concatenate([d(self.k[e:e + m, h]), d(self.r[e:e + m])], 1)
                ref = attention(d(self.q[a:a + n, h:h + 1]), k, d(self.v[e:e + m, h]), chain(n, m, self.causal), self.scale)
                check(o[a:a + n, h:h + 1], lse[a:a + n, h:h + 1], ref, f"request {b} (n {n}, m {m}) head {h}")
            a, e = a + n, e + m
        assert torch.all(self.od[a:] == 77.0) and torch.all(self.od[:, self.heads:] == 77.0) and torch.all(self.lse[a:] == 77.0)
        assert torch.all(self.od[:, :, 128:] == 77.0)


@pytest.mark.parametrize("n", [1, 63, 64, 65, 127, 128, 129, 256, 257, 600])
@pytest.mark.parametrize("before", [0, 1, 100, 700])
def test_lengths(n, before):
    Case([n], [n + before], heads=1, seed=n).check()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens,kv_lens", [([5, 300, 1], [5, 300, 1]), ([130, 0, 70], [700, 9, 70]),
                                            ([3, 4], [0, 2]), ([300, 1], [140, 3]), ([1] * 50, list(range(1, 51)))])
@pytest.mark.parametrize("heads", [1, 3, 16])
def test_batches(q_lens, kv_lens, causal, heads):
    """Empty requests, requests with fewer keys than rows (their first rows see nothing), none at all."""
    Case(q_lens, kv_lens, heads, causal, seed=heads, pad=heads % 2).check()


def test_no_keys_at_all():
    c = Case([3, 2], [0, 0])
    o, lse = c.run()
    assert int(c.err.item()) == 0 and np.all(o == 0) and np.all(np.isneginf(lse))
    empty = torch.empty(0, 2, 128, dtype=torch.bfloat16, device=DEV)
    c.args = B.attn_expanded_args(c.qd[:, :, :192], empty, torch.empty(0, 64, dtype=torch.bfloat16, device=DEV), empty,
                                  c.od, c.cu, c.cu_kv, 3, 0, 0.1, lse=c.lse, workspace=c.ws, err_flag=c.err)
    o, lse = c.run()
    assert int(c.err.item()) == 0 and np.all(o == 0) and np.all(np.isneginf(lse))


@pytest.mark.parametrize("max_ctas", [0, 1, 2, 7])
def test_splits(max_ctas):
    Case([1, 300], [3000, 1500], heads=2).check(max_ctas=max_ctas)
    Case([40, 2], [2000, 900], heads=1, causal=False).check(max_ctas=max_ctas)


def test_long_one_row_over_the_whole_gpu():
    Case([1], [30011], heads=1).check()


def test_same_bits_every_time():
    c = Case([500, 20], [900, 3000], heads=4)
    a = [x.copy() for x in c.run()]
    for _ in range(3):
        b = c.run()
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (1e-4, 1.0), (8.0, 1e-6), (1.0, 20.0)])
def test_ranges(std, scale):
    Case([70, 200], [400, 200], std=std, scale=scale).check()


def test_loose_bounds_shared_rows_and_no_lse():
    c = Case([9, 130], [50, 300], heads=5, pad=1)
    c.args = c.make_args(4000, 9000)
    c.check()
    c.args = c.make_args(lse=False)
    o, lse = c.run()
    assert np.all(lse == 77.0)
    c = Case([4, 2], [10, 20], heads=3)
    c.q[:] = c.q[:1, :1]
    one = c.q[:1, :1].to(DEV).expand(9, 3, 192)
    c.args = B.attn_expanded_args(one, c.kv[:, :, :128], c.rd, c.kv[:, :, 128:], c.od, c.cu, c.cu_kv, 4, 20, c.scale,
                                  lse=c.lse, workspace=c.ws, err_flag=c.err)
    c.check()


def test_bad_lengths():
    for q_lens, kv_lens, kw in (([3, 2], [8, 9], dict(max_q=2)), ([3, 2], [20, 9], dict(max_kv=10))):
        c = Case(q_lens, kv_lens)
        c.args = c.make_args(**kw)
        c.run()
        assert int(c.err.item()) == 7 and torch.all(c.od[:3] == 77.0) and not torch.any(c.od[3:5] == 77.0)
    c = Case([3, 2], [8, 9])
    c.cu_kv[2] = 1000  # past the keys there are
    c.args = c.make_args(max_kv=4000)
    c.run()
    assert int(c.err.item()) == 7 and torch.all(c.od[3:] == 77.0) and not torch.any(c.od[:3] == 77.0)


def test_another_stream_and_a_graph():
    c = Case([200, 100], [900, 333], heads=3)
    want = c.run()[0].copy()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        B.moe_attn_expanded(c.args)
    for _ in range(3):
        c.od.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(c.od[:300].double().cpu().numpy(), want)
    assert int(c.err.item()) == 0


def test_first_cta_gives_up():
    c = Case([300, 1], [3000, 500])
    want = c.run()[0].copy()
    B.moe_debug_inject_wait(True, 2_000_000)
    try:
        c.run()
    finally:
        B.moe_debug_inject_wait(False)
    assert int(c.err.item()) == 8 and int(c.ws[:4096].count_nonzero().item()) == 0
    c.err.zero_()
    assert np.array_equal(c.run()[0], want) and int(c.err.item()) == 0


def test_both_forms_agree():
    """Keys and values projected from latent vectors, and the projections absorbed into queries and outputs."""
    g = torch.Generator(device=DEV).manual_seed(0)
    rand = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.float64)
    H, n, kv, page = 4, 40, 150, 64
    latent, rope, q = rand(kv, 512).bfloat16().double(), rand(kv, 64).bfloat16(), rand(n, H, 192)
    wk, wv = rand(H, 512, 128) * 512**-0.5, rand(H, 512, 128) * 512**-0.5
    pool = torch.full((3, page, 576), float("nan"), dtype=torch.bfloat16, device=DEV)
    cache = B.latent_cache(pool)
    slots = torch.arange(kv, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_latent_write(cache, latent.bfloat16(), rope, slots, err_flag=err)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    k, v = (torch.einsum("sl,hld->shd", latent, w).bfloat16() for w in (wk, wv))
    o = torch.empty(n, H, 128, dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(B.moe_attn_expanded_workspace_size(H), dtype=torch.uint8, device=DEV)
    B.moe_attn_expanded(B.attn_expanded_args(q.bfloat16(), k, rope, v, o, i32([0, n]), i32([0, kv]), n, kv, 192**-0.5,
                                             workspace=ws, err_flag=err))
    qa = torch.cat([torch.einsum("nhd,hld->nhl", q.bfloat16().double()[..., :128], wk), q.bfloat16().double()[..., 128:]], 2)
    ol = torch.empty(n, H, 512, dtype=torch.bfloat16, device=DEV)
    B.moe_attn_latent(cache, B.attn_latent_args(qa.bfloat16(), ol, i32([0, n]), i32([kv]), i32([[0, 1, 2]]), n, kv,
                                                192**-0.5, workspace=ws, err_flag=err))
    oa = torch.einsum("nhl,hld->nhd", ol.double(), wv)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # keys and absorbed queries are rounded at different places: a score of size up to 5 is off by about 2^-9 of
    # the root of its 192 (576) products' squares, under 0.02, and so are o's parts; o is an average of |v| ~ 1
    assert (o.double() - oa).abs().max().item() <= 0.1 and (o.double() - oa).abs().mean().item() <= 0.01
