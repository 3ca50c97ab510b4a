"""Latent attention (absorbed form) on the GPU against a plain implementation in 64 bits: head counts, lengths,
page sizes, masks, trees, strides, splits over CTAs, and what must not reach a result."""
import numpy as np
import pytest
import torch

from latent_ref import attention, branches, chain, check, random_tree
from moe_expert_dispatch_route_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
L, R, D = 512, 64, 576


class Case:
    """A batch with its cache; every cached number that no row may see is NaN."""

    def __init__(self, q_lens, kv_lens, heads=16, page=64, causal=True, window=0, tree=False, seed=0, order="pages",
                 q_pad=0, scale=192**-0.5, std=1.0, spare=0):
        rng = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.heads, self.scale = q_lens, kv_lens, heads, scale
        self.causal, self.window = causal, window
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + 2
        width = max(max(need), 1)
        perm = rng.permutation(pages)
        table = np.full((len(kv_lens), width), -7, dtype=np.int32)  # never looked at past a request's pages
        pool = torch.full((pages, page, D), float("nan"), dtype=torch.bfloat16)
        self.keys, self.seen, bits = [], [], []
        at = 0
        for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
            mine = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine
            val = torch.tensor(rng.standard_normal((kv, D)) * std).to(torch.bfloat16)
            if tree:
                mask = random_tree(rng, n)
                bits.append(mask | np.uint64(1 << n if n < 64 else 0))  # a bit past the request's tokens counts for nothing
                self.seen.append(branches(mask, n, kv))
            else:
                self.seen.append(chain(n, kv, causal, window))
            some = self.seen[-1].any(0) if n else np.zeros(kv, dtype=bool)
            for j in np.flatnonzero(some):
                pool[mine[j // page], j % page] = val[j]
            for i in range(need[b]):  # pages already given back
                if not some[i * page:(i + 1) * page].any():
                    table[b, i] = -1
            self.keys.append(val.double().numpy())
        T = sum(q_lens)
        self.q = torch.tensor(rng.standard_normal((T, heads, D))).to(torch.bfloat16)
        wide = torch.full((pages, page, D + spare), float("nan"), dtype=torch.bfloat16, device=DEV)
        if order == "tokens":
            wide = wide.transpose(0, 1).contiguous().transpose(0, 1)
        wide[:, :, :D] = pool.to(DEV)
        self.pool = wide
        self.cache = B.latent_cache(wide[:, :, :D])
        self.qd = torch.zeros(T, heads + q_pad, D + 8 * q_pad, dtype=torch.bfloat16, device=DEV)
        self.qd[:, :heads, :D] = self.q.to(DEV)
        self.od = torch.full((T + 2, heads + q_pad, L + 8 * q_pad), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((T, heads), 77.0, device=DEV)
        self.cu = torch.tensor([0] + np.cumsum(q_lens).tolist(), dtype=torch.int32, device=DEV)
        self.kv = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        self.table = torch.tensor(table, device=DEV)
        self.tree = torch.from_numpy(np.concatenate(bits).view(np.int64)).to(DEV) if tree else None
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.zeros(B.moe_attn_latent_workspace_size(self.cache, heads), dtype=torch.uint8, device=DEV)
        self.args = self.make_args()

    def make_args(self, **kw):
        a = dict(max_q=max(self.q_lens), max_kv=max(self.kv_lens), scale=self.scale, causal=self.causal,
                 window=self.window, lse=self.lse, workspace=self.ws, err_flag=self.err)
        a.update(kw)
        T = sum(self.q_lens)
        return B.attn_latent_args(self.qd[:, :self.heads, :D], self.od[:T, :self.heads, :L], self.cu, self.kv, self.table,
                                  **a)

    def run(self, **kw):
        self.od.fill_(77.0)
        self.lse.fill_(77.0)
        B.moe_attn_latent(self.cache, self.args, tree=self.tree, **kw)
        torch.cuda.synchronize()
        return self.od[:sum(self.q_lens), :self.heads, :L].double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self, **kw):
        o, lse = self.run(**kw)
        assert int(self.err.item()) == 0
        assert int(self.ws[:4096].count_nonzero().item()) == 0, "the counters are left zero"
        first = 0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            q = self.q[first:first + n].double().numpy()
            ref = attention(q, self.keys[b], self.keys[b][:, :L], self.seen[b], self.scale)
            check(o[first:first + n], lse[first:first + n], ref, f"request {b} (n {n}, kv {kv})")
            first += n
        T = sum(self.q_lens)
        assert torch.all(self.od[T:] == 77.0) and torch.all(self.od[:, self.heads:] == 77.0), "only o's rows are written"
        assert torch.all(self.od[:, :, L:] == 77.0)


@pytest.mark.parametrize("heads", [1, 2, 5, 16])
@pytest.mark.parametrize("kv", [1, 63, 64, 65, 129, 700])
def test_one_token(heads, kv):
    Case([1], [kv], heads=heads, seed=kv).check()


@pytest.mark.parametrize("heads", [17, 20, 32, 33, 40, 64, 65, 96, 97, 127, 128])
def test_heads(heads):
    Case([1, 2, 1], [100, 333, 64], heads=heads, seed=heads).check()
    Case([7, 1], [257, 128], heads=heads, seed=heads).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order,spare", [("pages", 0), ("tokens", 0), ("pages", 64)])
def test_pages_and_orders(page, order, spare):
    Case([1, 3, 2, 1], [5, 301, 64, 777], page=page, order=order, spare=spare, seed=page).check()


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([5, 0, 2], [5, 9, 130]), ([1, 1, 1], [0, 3, 0]),
                                             ([6, 4], [3, 4]), ([64, 1, 33], [64, 200, 500]), ([0, 0], [5, 0]),
                                             ([200], [450]), ([3] * 40, list(range(3, 43)))])
@pytest.mark.parametrize("heads", [8, 128])
def test_lengths(q_lens, kv_lens, heads):
    """Empty requests, caches shorter than the new tokens (their first rows see nothing), chunks."""
    if max(q_lens) == 0:
        c = Case(q_lens, kv_lens, heads=heads)
        c.run()
        return
    Case(q_lens, kv_lens, heads=heads).check()


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [0, 1, 50, 64, 200, 1 << 30])
def test_masks(causal, window):
    Case([4, 1, 70], [300, 513, 130], causal=causal, window=window, page=16, seed=window & 255).check()


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2, 6], [1, 200, 64]), ([64, 13, 1], [64, 500, 129]), ([33], [1000]),
                                            ([5, 64], [3, 40])])
@pytest.mark.parametrize("heads", [4, 16, 48, 128])
def test_trees(q_lens, kv_lens, heads):
    Case(q_lens, kv_lens, heads=heads, tree=True, seed=heads).check()


@pytest.mark.parametrize("heads,max_ctas", [(16, 0), (16, 1), (16, 7), (128, 0), (128, 1), (128, 5), (40, 3)])
def test_splits(heads, max_ctas):
    """Long requests over many CTAs, many over few, with and without a tree."""
    Case([1, 2], [5000, 3333], heads=heads, seed=1).check(max_ctas=max_ctas)
    Case([4, 1, 1, 2], [1500, 90, 1, 640], heads=heads, tree=True, seed=2).check(max_ctas=max_ctas)


def test_long_context_over_the_whole_gpu():
    Case([1], [40000], heads=16, seed=3).check()
    Case([1], [20011], heads=128, seed=4).check()


def test_same_bits_every_time_and_any_grid_of_a_whole_tile():
    c = Case([3, 2, 1], [3000, 50, 700], heads=64)
    a = [x.copy() for x in c.run()]
    for _ in range(3):
        b = c.run()
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_strides_spare_rows_and_loose_bounds():
    c = Case([2, 5], [100, 300], heads=24, q_pad=3)
    c.check()
    c.args = c.make_args(max_q=1000, max_kv=5000)
    c.check()
    q = c.qd[:1, :1, :D].expand(7, 24, D)  # all rows the same
    c.q = q.cpu()
    c.args = B.attn_latent_args(q, c.od[:7, :24, :L], c.cu, c.kv, c.table, 5, 300, c.scale, lse=c.lse, workspace=c.ws,
                                err_flag=c.err)
    c.check()


@pytest.mark.parametrize("std,scale", [(30.0, 1.0), (1e-4, 1.0), (8.0, 1e-6), (1.0, 20.0)])
def test_ranges(std, scale):
    """Probabilities on one key, on all alike, and maxima that move often."""
    Case([1, 3, 2], [700, 350, 65], heads=20, std=std, scale=scale).check()


def test_rising_maximum():
    """Keys sorted by their score: the running maximum moves with every tile."""
    c = Case([1], [1500], heads=1, seed=9)
    k = c.keys[0]
    order = np.argsort(k @ c.q[0, 0].double().numpy())
    c.keys[0] = k[order] * np.linspace(0.1, 12, 1500)[:, None]
    c.keys[0] = torch.tensor(c.keys[0]).to(torch.bfloat16).double().numpy()
    flat = torch.tensor(c.keys[0]).to(torch.bfloat16).to(DEV)
    for j in range(1500):
        c.pool[int(c.table[0, j // 64]), j % 64, :D] = flat[j]
    c.check()


def test_bad_lengths_and_pages():
    c = Case([1, 2], [100, 200], heads=8)
    c.kv[0] = 5000  # more than the table has pages for, and than max_kv
    c.run()
    assert int(c.err.item()) == 7 and torch.all(c.od[0] == 77.0) and not torch.any(c.od[1:3, :8, :L] == 77.0)
    c = Case([1, 2], [100, 200], heads=8)
    c.table[1, 0] = 10**6
    c.run()
    assert int(c.err.item()) == 7 and torch.isfinite(c.od[:3].float()).all()
    c = Case([3, 2], [100, 200], heads=8)
    c.args = c.make_args(max_q=2)
    c.run()
    assert int(c.err.item()) == 7 and torch.all(c.od[:3] == 77.0) and not torch.any(c.od[3:5, :8, :L] == 77.0)


def test_another_stream_and_a_graph():
    c = Case([1, 4], [900, 333], heads=128)
    want = [x.copy() for x in c.run()]
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        B.moe_attn_latent(c.cache, c.args)
    for _ in range(3):
        c.od.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(c.od[:5, :128, :L].double().cpu().numpy(), want[0])
    assert int(c.err.item()) == 0


@pytest.mark.parametrize("heads", [16, 128])
def test_first_cta_gives_up(heads):
    """A bounded wait that runs out: the call reports it, counts its parts and leaves the workspace ready."""
    c = Case([1, 1], [3000, 500], heads=heads)
    want = [x.copy() for x in c.run()]
    B.moe_debug_inject_wait(True, 2_000_000)
    try:
        c.run()
    finally:
        B.moe_debug_inject_wait(False)
    assert int(c.err.item()) == 8 and int(c.ws[:4096].count_nonzero().item()) == 0
    c.err.zero_()
    got = c.run()
    assert np.array_equal(got[0], want[0]) and int(c.err.item()) == 0
