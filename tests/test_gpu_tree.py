"""moe_attn_tree on the GPU against a plain implementation in 64 bits: both kernels, both cache types."""
import numpy as np
import pytest
import torch

from latent_ref import attention, branches, check, random_tree
from moe_expert_dispatch_route_gb300 import binding as B
from serve_ref import E4M3, dequantise

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    def __init__(self, q_lens, kv_lens, Hq=8, H=2, D=128, page=16, dtype="bf16", seed=0, bits=None):
        rng = np.random.default_rng(seed)
        self.q_lens, self.kv_lens, self.Hq, self.H, self.D = q_lens, kv_lens, Hq, H, D
        need = [-(-n // page) for n in kv_lens]
        pages = sum(need) + 2
        perm = rng.permutation(pages)
        table = np.full((len(kv_lens), max(max(need), 1)), -7, dtype=np.int32)
        fp8 = dtype == "e4m3"
        if fp8:
            pool = np.full((2, pages, H, page, D), 0x7F, dtype=np.uint8)
            scales = np.full((2, pages, H, page), 255, dtype=np.uint8)
        else:
            pool = torch.full((2, pages, H, page, D), float("nan"), dtype=torch.bfloat16)
        self.k, self.v, self.seen, masks = [], [], [], []
        at = 0
        for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
            mine = perm[at:at + need[b]]
            at += need[b]
            table[b, :need[b]] = mine
            val = rng.standard_normal((2, kv, H, D))
            if fp8:
                codes = torch.tensor(val * 100).clamp(-448, 448).to(E4M3).view(torch.uint8).numpy()
                sc = rng.integers(118, 123, size=(2, kv, H)).astype(np.uint8)
                val = np.stack([dequantise(codes[i], sc[i]) for i in range(2)])
            else:
                val = torch.tensor(val).to(torch.bfloat16)
            for j in range(kv):
                pool[:, mine[j // page], :, j % page] = codes[:, j] if fp8 else val[:, j]
                if fp8:
                    scales[:, mine[j // page], :, j % page] = sc[:, j]
            mask = random_tree(rng, n) if bits is None else np.array(bits, dtype=np.uint64)
            masks.append(mask)
            self.seen.append(branches(mask, n, kv))
            val = val if fp8 else val.double().numpy()
            self.k.append(val[0])
            self.v.append(val[1])
        T = sum(q_lens)
        self.q = torch.tensor(rng.standard_normal((T, Hq, D))).to(torch.bfloat16)
        pool = torch.as_tensor(pool).to(DEV)
        self.keep = torch.tensor(scales, device=DEV) if fp8 else None
        self.pool = pool.view(E4M3) if fp8 else pool
        self.cache = B.kv_cache(self.pool[0], self.pool[1], *((self.keep[0], self.keep[1]) if fp8 else ()))
        self.qd = self.q.to(DEV)
        self.od = torch.full((T + 1, Hq, D), 77.0, dtype=torch.bfloat16, device=DEV)
        self.lse = torch.full((T, Hq), 77.0, device=DEV)
        self.cu = torch.tensor([0] + np.cumsum(q_lens).tolist(), dtype=torch.int32, device=DEV)
        self.kv = torch.tensor(kv_lens, dtype=torch.int32, device=DEV)
        self.table = torch.tensor(table, device=DEV)
        self.tree = torch.from_numpy(np.concatenate(masks).view(np.int64)).to(DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.ws = torch.zeros(B.moe_attn_workspace_size(self.cache, Hq), dtype=torch.uint8, device=DEV)
        self.args = B.attn_args(self.qd, self.od[:T], self.cu, self.kv, self.table, max(q_lens), max(kv_lens), D**-0.5,
                                lse=self.lse, workspace=self.ws, err_flag=self.err)

    def run(self, **kw):
        self.od.fill_(77.0)
        self.lse.fill_(77.0)
        B.moe_attn_tree(self.cache, self.args, self.tree, **kw)
        torch.cuda.synchronize()
        return self.od[:-1].double().cpu().numpy(), self.lse.double().cpu().numpy()

    def check(self, **kw):
        o, lse = self.run(**kw)
        assert int(self.err.item()) == 0 and int(self.ws[:4096].count_nonzero().item()) == 0
        assert torch.all(self.od[-1] == 77.0)
        G, first = self.Hq // self.H, 0
        for b, (n, kv) in enumerate(zip(self.q_lens, self.kv_lens)):
            q = self.q[first:first + n].double().numpy()
            for h in range(self.H):
                ref = attention(q[:, h * G:(h + 1) * G], self.k[b][:, h], self.v[b][:, h], self.seen[b], self.D**-0.5)
                check(o[first:first + n, h * G:(h + 1) * G], lse[first:first + n, h * G:(h + 1) * G], ref,
                      f"request {b} (n {n}, kv {kv}) head {h}")
            first += n


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 2), (7, 1), (32, 4)])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2, 4], [1, 60, 300]), ([8, 5, 1], [8, 130, 257]),
                                            ([64, 13], [64, 400]), ([33, 1, 64], [200, 77, 129])])
def test_trees(dtype, D, Hq, H, q_lens, kv_lens):
    Case(q_lens, kv_lens, Hq, H, D, dtype=dtype, seed=Hq).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("max_ctas", [0, 1, 7])
def test_pages_and_splits(dtype, page, max_ctas):
    Case([6, 3], [2500, 90], page=page, dtype=dtype, seed=page).check(max_ctas=max_ctas)
    Case([50, 3, 17], [1800, 90, 17], page=page, dtype=dtype, seed=page).check(max_ctas=max_ctas)


@pytest.mark.parametrize("q_lens,kv_lens", [([5, 0, 2], [3, 9, 1]), ([64, 40], [30, 10]), ([2, 3], [0, 0])])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_caches_shorter_than_the_tree(q_lens, kv_lens, dtype):
    Case(q_lens, kv_lens, dtype=dtype).check()


def test_any_mask_and_bits_past_the_tokens():
    """A token may see later ones; it sees itself without being asked; bits past the request's count for nothing."""
    Case([4], [100], bits=[0b1010, 0b0001, 0, 0b0111]).check()
    full = (1 << 64) - 1
    Case([3], [50], bits=[full, full ^ 7, 1 << 63]).check()
    Case([30], [50], Hq=16, H=1, bits=[full] * 30).check()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("n", [5, 60])
def test_a_chain_is_a_tree(n, dtype):
    """The same bits as causal attention, where the kernel's tiles are the same."""
    c = Case([n, n], [700, 300], dtype=dtype, bits=[(1 << (i + 1)) - 1 for i in range(n)])
    o, lse = (x.copy() for x in c.run())
    c.od.fill_(0)
    B.moe_attn_paged(c.cache, c.args)
    torch.cuda.synchronize()
    assert np.abs(c.od[:-1].double().cpu().numpy() - o).max() <= 2.0**-6  # tiles may be cut elsewhere
    assert np.abs(c.lse.double().cpu().numpy() - lse).max() <= 1e-4


def test_graph():
    c = Case([9, 4], [500, 60])
    want = c.run()[0].copy()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        B.moe_attn_tree(c.cache, c.args, c.tree)
    c.od.fill_(0)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(c.od[:-1].double().cpu().numpy(), want)
