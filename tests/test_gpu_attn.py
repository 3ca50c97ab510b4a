"""Paged attention on the GPU against a plain implementation in 64 bits: types, head layouts,
lengths, page sizes, masks, strides, splits over CTAs, and what must not reach a result."""
import math

import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from serve_ref import E4M3, attention, dequantise

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    """A batch with its cache; everything that no row may see holds NaN."""

    def __init__(self, q_lens, kv_lens, Hq=8, H=2, D=128, page=16, dtype="bf16", causal=True, window=0, seed=0,
                 order="hnd", q_pad=0, scale=None, std=1.0):
        rng = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.Hq, self.H, self.D = q_lens, kv_lens, Hq, H, D
        self.causal, self.window = causal, window
        self.scale = 1 / math.sqrt(D) if scale is None else scale
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + 2
        width = max(max(need), 1)
        perm = rng.permutation(pages)
        table = np.full((len(kv_lens), width), -7, dtype=np.int32)  # never looked at past a request's pages
        fp8 = dtype == "e4m3"
        if fp8:
            pool = np.full((2, pages, H, page, D), 0x7F, dtype=np.uint8)
            scales = np.full((2, pages, H, page), 255, dtype=np.uint8)
        else:
            pool = torch.full((2, pages, H, page, D), float("nan"), dtype=torch.bfloat16)
        self.k, self.v = [], []
        at = 0
        for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
            mine = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine
            # tokens left of every row's window are stale too
            first = max(0, kv - n - window + 1) if window and causal else 0
            val = rng.standard_normal((2, kv, H, D)) * std
            if fp8:
                codes = torch.tensor(val * 100).clamp(-448, 448).to(E4M3).view(torch.uint8).numpy()
                sc = rng.integers(118, 123, size=(2, kv, H)).astype(np.uint8)
                val = np.stack([dequantise(codes[i], sc[i]) for i in range(2)])
            else:
                val = torch.tensor(val).to(torch.bfloat16)
            for j in range(first, kv):
                if fp8:
                    pool[:, mine[j // page], :, j % page] = codes[:, j]
                    scales[:, mine[j // page], :, j % page] = sc[:, j]
                else:
                    pool[:, mine[j // page], :, j % page] = val[:, j]
            for p in range(first // page):  # pages already given back
                table[b, p] = -1
            val = val if fp8 else val.double().numpy()
            self.k.append(val[0])
            self.v.append(val[1])
        T = sum(q_lens)
        self.q = torch.tensor(rng.standard_normal((T, Hq, D))).to(torch.bfloat16)
        pool = torch.as_tensor(pool).to(DEV)
        if fp8:
            pool = pool.view(E4M3)
            sc = torch.tensor(scales, device=DEV)
        a, b = {"hnd": (0, 0), "nhd": (2, 3), "head first": (1, 2)}[order]
        self.pool = pool.transpose(a, b).contiguous().transpose(a, b)
        self.cache = B.kv_cache(self.pool[0], self.pool[1], *((sc[0], sc[1]) if fp8 else ()))
        self.keep = sc if fp8 else None
        # q and o as parts of wider buffers
        self.qd = torch.zeros(T, Hq + q_pad, D, dtype=torch.bfloat16, device=DEV)
        self.qd[:, :Hq] = self.q.to(DEV)
        self.od = torch.full((T, Hq + q_pad, D), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((T, Hq), 77.0, device=DEV)
        self.cu = torch.tensor([0] + np.cumsum(q_lens).tolist(), dtype=torch.int32, device=DEV)
        self.kv = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        self.table = torch.tensor(table, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.zeros(B.moe_attn_workspace_size(self.cache, Hq), dtype=torch.uint8, device=DEV)
        self.args = self.make_args()

    def make_args(self, **kw):
        a = dict(max_q=max(self.q_lens), max_kv=max(self.kv_lens), scale=self.scale, causal=self.causal,
                 window=self.window, lse=self.lse, workspace=self.ws, err_flag=self.err)
        a.update(kw)
        return B.attn_args(self.qd[:, :self.Hq], self.od[:, :self.Hq], self.cu, self.kv, self.table, **a)

    def run(self, **kw):
        self.od.fill_(77.0)
        self.lse.fill_(77.0)
        B.moe_attn_paged(self.cache, self.args, **kw)
        torch.cuda.synchronize()
        return self.od[:, :self.Hq].double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self, **kw):
        """bf16's unit roundoff is 2^-8 (8 significant bits).  |o - exact| <= 2^-8 |o| (its rounding)
        + 2^-8 sum p|v| (that of the probabilities) and 2^-12
        of that sum for scores held in fp32: a score's error is at most D * 2^-24 * scale * sum |q k|,
        under 6e-5 at these sizes, the same relative change of each p.  lse: twice that bound."""
        o, lse = self.run(**kw)
        assert int(self.err.item()) == 0
        assert int(self.ws[:4096].count_nonzero().item()) == 0, "the counters are left zero"
        first = 0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            q = self.q[first:first + n].double().numpy()
            ro, rl, mag = attention(q, self.k[b], self.v[b], kv, self.scale, self.causal, self.window)
            go, gl = o[first:first + n], lse[first:first + n]
            empty = np.isneginf(rl)
            assert np.array_equal(np.isneginf(gl), empty), f"request {b}: rows that see nothing"
            assert np.all(go[empty] == 0)
            bad = np.abs(go - ro) > 2.0**-8 * np.abs(ro) + (2.0**-8 + 2.0**-12) * mag + 1e-30
            assert not bad.any() and np.isfinite(go).all(), \
                f"request {b} (n {n}, kv {kv}): {bad.sum()} of {bad.size} outputs off, first {np.argwhere(bad)[:3]}"
            assert np.abs(gl[~empty] - rl[~empty]).max(initial=0) <= 1.2e-4, f"request {b}: lse"
            first += n
        assert torch.all(self.od[:, self.Hq:] == 77.0), "only o's heads are written"


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[1, 2, 1], [50, 200, 3]])
def test_loose_bounds_and_spare_rows(dtype, q_lens):
    """max_q and max_kv far above the lengths (so that a kernel for many rows gets few), a wider block
    table, rows of q and o past the last request, and heads apart from each other in q and o."""
    c = Case(q_lens, [90, 300, 257], dtype=dtype)
    T, Hq, D = c.qd.shape
    wide = lambda t, fill: torch.full((T + 5, Hq, 2 * D), fill, dtype=torch.bfloat16, device=DEV)
    q, o = wide(c.qd, float("nan")), wide(c.od, 77.0)
    q[:T, :, :D] = c.qd
    table = torch.full((3, 40), -9, dtype=torch.int32, device=DEV)
    table[:, :c.table.shape[1]] = c.table
    lse = torch.full((T + 5, Hq), 77.0, device=DEV)
    args = B.attn_args(q[:, :, :D], o[:, :, :D], c.cu, c.kv, table, 1000, 600, c.scale, lse=lse, workspace=c.ws,
                       err_flag=c.err)
    B.moe_attn_paged(c.cache, args)
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0 and torch.all(o[T:] == 77.0) and torch.all(o[:, :, D:] == 77.0)
    assert torch.all(lse[T:] == 77.0)
    c.od[:, :], c.lse[:, :] = o[:T, :, :D], lse[:T]
    c.run, go = (lambda **kw: go), (c.od.double().cpu().numpy(), c.lse.double().cpu().numpy())
    c.check()


KV_EDGES = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 1000]


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(1, 1), (8, 8), (8, 2), (6, 2), (32, 4), (5, 1), (64, 1)])
def test_decode(dtype, D, Hq, H):
    Case([1] * len(KV_EDGES), KV_EDGES, Hq=Hq, H=H, D=D, dtype=dtype).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["hnd", "nhd", "head first"])
def test_pages_and_orders(page, dtype, order):
    Case([1, 3, 1, 2], [5, 300, 513, 700], page=page, dtype=dtype, order=order, q_pad=3).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(4, 4), (8, 2), (14, 2), (24, 3), (20, 1)])
def test_drafts(dtype, D, Hq, H):
    Case([2, 5, 1, 4, 3, 5], [2, 5, 40, 129, 300, 517], Hq=Hq, H=H, D=D, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 1), (7, 1), (3, 1), (48, 1)])
def test_chunks(dtype, D, Hq, H):
    Case([1, 130, 33, 257, 64], [1, 130, 100, 400, 333], Hq=Hq, H=H, D=D, dtype=dtype, page=32).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [4, 1, 3], [40, 200, 1]])
@pytest.mark.parametrize("window", [1, 5, 128, 150])
def test_windows(dtype, q_lens, window):
    Case(q_lens, [300, 700, 129], window=window, dtype=dtype).check()


@pytest.mark.parametrize("q_lens", [[1, 4, 0], [150, 33, 5]])
def test_the_widest_window(q_lens):
    """A window past every position is none, also for rows that stand before the first token."""
    c = Case(q_lens, [200, 3, 129])
    o, lse = c.run()
    c.args = c.make_args(window=2**31 - 1)
    o2, lse2 = c.run()
    assert np.array_equal(o, o2) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[1, 2, 3], [70, 5, 150]])
@pytest.mark.parametrize("window", [0, 20])
def test_not_causal(dtype, q_lens, window):
    Case(q_lens, [200, 64, 150], causal=False, window=window, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("scale_up", [1, 30])
def test_rows_that_see_nothing(dtype, causal, scale_up):
    # no cached token; fewer cached tokens than rows (the first rows stand before them); no rows
    q, kv = [2, 5, 0, 3, 1], [0, 3, 40, 3, 0]
    Case([n * scale_up for n in q], kv, dtype=dtype, causal=causal).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("max_ctas", [1, 2, 3, 7, 31])
def test_splits_over_ctas(dtype, max_ctas):
    """Ranges that begin and end anywhere in a tile, tiles over many CTAs."""
    Case([1, 4, 2], [1500, 130, 900], Hq=4, H=1, dtype=dtype).check(max_ctas=max_ctas)
    Case([150, 1, 40], [700, 900, 40], Hq=4, H=2, dtype=dtype).check(max_ctas=max_ctas)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 100])
def test_one_long_context(dtype, n):
    """One tile of rows over the whole GPU."""
    Case([n], [20000], Hq=2, H=1, dtype=dtype, page=64).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("max_ctas", [9, 37, 1000])
def test_tiles_of_many_parts(dtype, D, max_ctas):
    """Few query tiles over many CTAs, whose parts are summed in groups of groups."""
    Case([130, 40], [6000, 2500], Hq=8, H=2, D=D, dtype=dtype, page=64).check(max_ctas=max_ctas)


def test_many_requests():
    rng = np.random.default_rng(3)
    n = 700
    kv = rng.integers(1, 80, size=n).tolist()
    Case([1] * n, kv, Hq=2, H=1, D=64).check()


def test_large_scores_and_a_large_scale():
    """Running maxima that jump: keys far apart, scores of a few hundred."""
    c = Case([1, 3], [777, 300], std=8.0, scale=1.0, seed=5)
    o, lse = c.run()
    first = 0
    for b, (n, kv) in enumerate(zip(c.q_lens, c.kv_lens)):
        ro, rl, mag = attention(c.q[first:first + n].double().numpy(), c.k[b], c.v[b], kv, 1.0)
        # scores up to ~400 held in fp32: errors up to 400 * 2^-24 * 128 = 3e-3 of each p
        assert (np.abs(o[first:first + n] - ro) <= 2.0**-8 * np.abs(ro) + (2.0**-8 + 4e-3) * mag).all()
        assert np.abs(lse[first:first + n] - rl).max() <= 4e-3
        first += n


@pytest.mark.parametrize("n", [1, 20, 70])
@pytest.mark.parametrize("what", ["q0", "tiny q", "huge q", "far scales"])
def test_e4m3_ranges(n, what):
    """Rows of zeros and of extreme size, and key and value scales far from 1 and from each other:
    what fp16 operands have to be scaled for.  An error may be 2^-31 of the largest number of its
    kind (see the kernels), under the bound by far for these."""
    c = Case([n, n], [300, 200], dtype="e4m3", seed=7)
    f = {"q0": 0.0, "tiny q": 2.0**-120, "huge q": 2.0**100, "far scales": 1.0}[what]
    c.q = (c.q.float() * f).to(torch.bfloat16)
    c.qd[:, :c.Hq] = c.q.to(DEV)
    if what == "huge q":  # against keys as small
        c.keep[0] = torch.where(c.keep[0] == 255, c.keep[0], c.keep[0] - 90)
        c.k = [k * 2.0**-90 for k in c.k]
        c.scale = c.scale * 2.0**-10
        c.args = c.make_args()
    if what == "far scales":
        rng = np.random.default_rng(1)
        for b, kv in enumerate(c.kv_lens):
            for j in range(kv):
                page, at = int(c.table[b, j // 16]), j % 16
                for i, t in ((0, c.k), (1, c.v)):
                    up = int(rng.integers(-20, 21)) if i else -int(rng.integers(0, 30))
                    c.keep[i, page, :, at] += up
                    t[b][j] *= 2.0**up
    c.check()


@pytest.mark.parametrize("q_lens", [[1, 2], [150, 33]])
def test_the_same_bits_every_time(q_lens):
    c = Case(q_lens, [5000, 3000], Hq=8, H=2, page=64)
    o, lse = c.run()
    for _ in range(5):
        o2, lse2 = c.run()
        assert np.array_equal(o, o2) and np.array_equal(lse, lse2)


@pytest.mark.parametrize("q_lens", [[1, 2], [150, 33]])
def test_other_stream_and_graph(q_lens):
    c = Case(q_lens, [500, 300], Hq=8, H=2, page=64)
    want, lse = c.run()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, lse2 = c.run(stream=s)
    assert np.array_equal(want, got) and np.array_equal(lse, lse2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        B.moe_attn_paged(c.cache, c.args, stream=torch.cuda.current_stream())
    for _ in range(3):
        c.od.fill_(5.0)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(want, c.od[:, :c.Hq].double().cpu().numpy())


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [1, 70])
def test_nan_where_a_row_sees_it(dtype, n):
    """A NaN key or value makes the rows that see it NaN, and no other request's."""
    c = Case([n, n], [90, 200], dtype=dtype)
    page = int(c.table[0, 0])
    if dtype == "bf16":
        c.pool[0, page, 0, 3, 5] = float("nan")
    else:
        c.keep[0, page, 0, 3] = 255
    o, _ = c.run()
    assert np.isnan(o[:n, :4]).all() and np.isfinite(o[:n, 4:]).all() and np.isfinite(o[n:]).all()


@pytest.mark.parametrize("n", [1, 70])
def test_errors_found_on_the_device(n):
    c = Case([n, n], [200, 300])
    want, _ = c.run()
    c.table[0, 2] = c.pool.shape[1] + 5
    o, _ = c.run()
    assert int(c.err.item()) == 7 and np.array_equal(o[n:], want[n:]) and np.isfinite(o).all()
    for kw in (dict(max_q=n - 1) if n > 1 else dict(max_kv=299), dict(max_kv=250)):
        c = Case([n, n], [200, 300])
        c.args = c.make_args(**kw)
        o, _ = c.run()
        assert int(c.err.item()) == 7 and (o[n:] == 77.0).all(), "a refused request's rows are not written"
    c = Case([n, n], [200, 300])
    c.table = c.table[:, :13].contiguous()  # room for 208 tokens
    c.args = c.make_args()
    o, _ = c.run()
    assert int(c.err.item()) == 7 and (o[n:] == 77.0).all() and np.array_equal(o[:n], want[:n])


@pytest.mark.parametrize("n", [1, 70])
def test_a_bounded_wait_that_runs_out(n):
    c = Case([n, n], [200, 300])
    B.moe_debug_inject_wait(True, 1000000)
    try:
        c.run()
    finally:
        B.moe_debug_inject_wait(False)
    assert int(c.err.item()) == 8
    c.err.zero_()
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_lens", [[1, 3], [150, 33, 1]])
@pytest.mark.parametrize("shared", ["heads", "tokens", "both"])
def test_shared_query_rows(dtype, D, q_lens, shared):
    """q with a stride of 0: one row for all heads of a token, for all tokens, or for everything."""
    c = Case(q_lens, [300, 200, 64][:len(q_lens)], Hq=12, H=2, D=D, dtype=dtype)
    one = c.qd[:1 if shared != "heads" else None, :1 if shared != "tokens" else None].clone()
    c.qd = one.expand(*c.qd.shape)
    assert 0 in c.qd.stride()[:2]
    c.q = c.qd.cpu()
    c.args = c.make_args()
    c.check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("order", ["hnd", "nhd", "head first"])
def test_chunks_in_pages_and_orders(page, dtype, order):
    Case([70, 150, 1], [300, 513, 700], page=page, dtype=dtype, order=order, q_pad=3).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("requests", [40, 600])
def test_chunks_of_many_requests(dtype, requests):
    """More requests than a warp's lanes, and than the CTA's threads: with several query tiles, with one, with no row
    and with rows that stand before the first token."""
    rng = np.random.default_rng(requests)
    q = rng.choice([0, 1, 5, 40, 90], size=requests, p=[0.2, 0.3, 0.3, 0.15, 0.05])
    q[0], q[requests // 2], q[-1] = 200, 0, 150
    kv = [int(n + rng.integers(0, 60)) if rng.random() < 0.9 else int(rng.integers(0, n + 1)) for n in q]
    Case([int(n) for n in q], kv, Hq=4, H=1, D=64, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens", [[1, 1, 1], [4, 1, 3], [40, 200, 1]])
@pytest.mark.parametrize("window", [1, 5, 128, 150])
def test_windows_of_64_columns(dtype, q_lens, window):
    Case(q_lens, [300, 700, 129], D=64, window=window, dtype=dtype).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 70])
@pytest.mark.parametrize("bad", [-1, 10**6])
def test_pages_outside_the_pool_read_as_zeros(dtype, D, n, bad):
    """A page outside the pool sets the error flag, and its tokens have keys and values of 0."""
    c = Case([n, n], [200, 300], D=D, dtype=dtype)
    c.table[0, 2] = bad
    c.k[0][32:48] = 0
    c.v[0][32:48] = 0
    c.run()
    assert int(c.err.item()) == 7
    c.err.zero_()
    run = c.run

    def no_error():
        out = run()
        c.err.zero_()
        return out

    c.run = no_error
    c.check()
