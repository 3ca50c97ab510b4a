"""Forms of latent attention that users meet and one kernel or the other has to take: sliding windows and no causal mask
on one CTA, every page size and pool order on pairs, bad pages and lengths on pairs, batches without new tokens, any
number of CTAs, calls beside each other, offsets past 32 bits."""
import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from test_gpu_expanded import Case as Expanded
from test_gpu_latent import D, DEV, L, Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [1, 50, 64, 200, 1 << 30])
@pytest.mark.parametrize("heads", [2, 8, 16])
def test_masks_on_one_cta(causal, window, heads):
    """Up to 64 rows a request; keys before the window are NaN, their pages given back."""
    Case([4, 1, 3], [300, 513, 130], heads=heads, causal=causal, window=window, page=16, seed=window & 255).check()
    Case([1, 1], [3001, 64], heads=heads, causal=causal, window=window, page=64, seed=heads).check(max_ctas=5)


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 33), (False, 100), (True, 700)])
@pytest.mark.parametrize("heads", [65, 128])
def test_masks_on_pairs_by_heads(causal, window, heads):
    Case([2, 1], [300, 1513], heads=heads, causal=causal, window=window, page=16, seed=window).check()


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order,spare", [("pages", 0), ("tokens", 0), ("pages", 64)])
@pytest.mark.parametrize("heads,q_lens", [(128, [1, 2, 1, 1]), (20, [4, 7, 1, 2])])
def test_pages_and_orders_on_pairs(page, order, spare, heads, q_lens):
    Case(q_lens, [5, 301, 64, 777], heads=heads, page=page, order=order, spare=spare, seed=page).check()
    Case(q_lens, [40, 301, 97, 500], heads=heads, page=page, order=order, window=70, seed=page).check()


@pytest.mark.parametrize("heads,n", [(128, 2), (20, 5)])
def test_bad_lengths_and_pages_on_pairs(heads, n):
    rows = lambda c, a, b: c.od[a:b, :heads, :L]
    c = Case([n, n], [100, 200], heads=heads)
    c.kv[0] = 5000  # more than the table has pages for, and than max_kv
    c.run()
    assert int(c.err.item()) == 7 and torch.all(rows(c, 0, n) == 77.0) and not torch.any(rows(c, n, 2 * n) == 77.0)
    for bad in (10**6, -1):
        c = Case([n, n], [100, 200], heads=heads)
        want = c.run()[0][:n]
        c.table[1, 0] = bad  # its tokens read as zeros
        c.run()
        assert int(c.err.item()) == 7 and torch.isfinite(rows(c, 0, 2 * n).float()).all()
        assert np.array_equal(rows(c, 0, n).double().cpu().numpy(), want)
    c = Case([n, n - 1], [100, 200], heads=heads)
    c.args = c.make_args(max_q=n - 1)
    c.run()
    assert int(c.err.item()) == 7 and torch.all(rows(c, 0, n) == 77.0) and not torch.any(rows(c, n, 2 * n - 1) == 77.0)


@pytest.mark.parametrize("heads", [16, 128])
def test_no_request_has_a_row(heads):
    """Rows of q that belong to no request: nothing is written."""
    c = Case([2, 1], [100, 70], heads=heads)
    c.cu.zero_()
    c.run()
    assert int(c.err.item()) == 0 and torch.all(c.od == 77.0) and torch.all(c.lse == 77.0)
    assert int(c.ws[:4096].count_nonzero().item()) == 0
    e = Expanded([3, 2], [8, 9])
    e.cu.zero_()
    e.run()
    assert int(e.err.item()) == 0 and torch.all(e.od == 77.0) and torch.all(e.lse == 77.0)
    assert int(e.ws[:4096].count_nonzero().item()) == 0


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_same_bits_on_any_number_of_ctas(heads):
    """Query tiles that no boundary of CTAs divides (256 keys and less)."""
    c = Case([3, 2, 1, 1], [250, 50, 129, 7], heads=heads)
    want = [x.copy() for x in c.run()]
    for n in (1, 2, 3, 7, 50):
        got = c.run(max_ctas=n)
        assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])
    e = Expanded([130, 2, 1], [256, 50, 129], heads=3)
    want = [x.copy() for x in e.run()]
    for n in (1, 2, 3, 7, 50):
        got = e.run(max_ctas=n)
        assert np.array_equal(want[0], got[0]) and np.array_equal(want[1], got[1])


@pytest.mark.parametrize("heads", [16, 128])
def test_two_calls_at_once(heads):
    """On streams of their own, a workspace each, one of them replayed from a graph."""
    cases = [Case([1, 3], [4000, 700], heads=heads, seed=s) for s in (1, 2)]
    want = [[x.copy() for x in c.run()] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=streams[0]):
        B.moe_attn_latent(cases[0].cache, cases[0].args)
    for c in cases:
        c.od.fill_(0)
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(streams[0]):
            g.replay()
        B.moe_attn_latent(cases[1].cache, cases[1].args, stream=streams[1])
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert np.array_equal(c.od[:4, :heads, :L].double().cpu().numpy(), w[0]) and int(c.err.item()) == 0


@pytest.mark.parametrize("heads", [16, 128])
def test_a_pool_past_31_bits(heads):
    """A cache of more than 2^31 numbers, written and read at its end."""
    pages = (1 << 31) // (64 * D) + 40
    pool = torch.empty(pages, 64, D, dtype=torch.bfloat16, device=DEV)
    c = Case([1, 2], [900, 70], heads=heads)
    want = c.run()[0].copy()
    moved = pages - 1 - torch.arange(c.pool.shape[0], device=DEV, dtype=torch.int32)
    cache = B.latent_cache(pool)
    flat = c.pool.view(-1, D)
    slots = (moved.long()[:, None] * 64 + torch.arange(64, device=DEV)).reshape(-1)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_latent_write(cache, flat[:, :L], flat[:, L:], slots, err_flag=err)
    assert int(err.item()) == 0 and torch.equal(pool[-1].view(torch.int16), c.pool[0].view(torch.int16))
    c.table = torch.where(c.table >= 0, moved[c.table.clamp(min=0).long()], -7)
    c.cache, c.args = cache, c.make_args()
    assert np.array_equal(c.run()[0], want) and int(c.err.item()) == 0


def test_rows_past_31_bits():
    """More than 2^31 numbers in q (absorbed), and in q and k (expanded): the last request's rows are those of a small call."""
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    requests, heads = 7400, 128
    T = 4 * requests
    q = torch.randn(4, heads, D, device=DEV).to(torch.bfloat16).repeat(requests, 1, 1)
    assert q.numel() > 1 << 31
    pool = torch.randn(4, 16, D, device=DEV).to(torch.bfloat16)
    o, err = torch.empty(T, heads, L, dtype=torch.bfloat16, device=DEV), i32([0])
    cache = B.latent_cache(pool)
    ws = torch.zeros(B.moe_attn_latent_workspace_size(cache, heads), dtype=torch.uint8, device=DEV)
    B.moe_attn_latent(cache, B.attn_latent_args(q, o, i32(range(0, T + 1, 4)), i32([60] * requests),
                                                i32([[2, 0, 3, 1]] * requests), 4, 60, 0.07, workspace=ws, err_flag=err))
    small = torch.empty(4, heads, L, dtype=torch.bfloat16, device=DEV)
    B.moe_attn_latent(cache, B.attn_latent_args(q[:4], small, i32([0, 4]), i32([60]), i32([[2, 0, 3, 1]]), 4, 60, 0.07,
                                                workspace=ws, err_flag=err))
    assert int(err.item()) == 0 and torch.equal(o.view(requests, 4, heads, L), small[None].expand(requests, -1, -1, -1))
    del q, o
    requests, n = 540, 256
    T = n * requests
    rand = lambda *s: torch.randn(*s, device=DEV).to(torch.bfloat16)
    one = [rand(n, heads, 192), rand(n, heads, 128), rand(n, 64), rand(n, heads, 128)]
    all_ = [t.repeat(requests, *[1] * (t.dim() - 1)) for t in one]
    assert all_[1].numel() > 1 << 31
    o, small = (torch.empty(rows, heads, 128, dtype=torch.bfloat16, device=DEV) for rows in (T, n))
    cu = i32(range(0, T + 1, n))
    B.moe_attn_expanded(B.attn_expanded_args(*all_, o, cu, cu, n, n, 0.07, workspace=ws, err_flag=err))
    B.moe_attn_expanded(B.attn_expanded_args(*one, small, cu[:2].contiguous(), cu[:2].contiguous(), n, n, 0.07, workspace=ws, err_flag=err))
    assert int(err.item()) == 0
    assert torch.equal(o.view(requests, n, heads, 128), small[None].expand(requests, -1, -1, -1))


@pytest.mark.parametrize("heads", [16, 128])
def test_rows_behind_the_last_request(heads):
    c = Case([2, 3], [100, 300], heads=heads)
    want = [x.copy() for x in c.run()]
    c.cu[2] = 2  # the second request has no new token: three rows of q are nobody's
    o, lse = c.run()
    assert int(c.err.item()) == 0 and np.all(o[2:] == 77.0) and np.all(lse[2:] == 77.0)
    assert np.array_equal(o[:2], want[0][:2]) and np.array_equal(lse[:2], want[1][:2])


@pytest.mark.parametrize("heads", [16, 128])
def test_a_request_full_of_nan_leaves_the_others_alone(heads):
    c = Case([1, 2, 1], [200, 100, 250], heads=heads)
    want = [x.copy() for x in c.run()]
    c.pool[c.table[1, :2].long()] = float("nan")
    c.qd[3] = float("inf")
    o, lse = c.run()
    assert int(c.err.item()) == 0 and np.isnan(o[1:]).all() and np.array_equal(o[:1], want[0][:1])
    c.qd[3] = 0.0
    o, lse = c.run()
    assert np.isnan(o[1:3]).all() and np.isfinite(o[3]).all() and np.array_equal(lse[0], want[1][0])
    for what in (float("nan"), float("inf")):
        e = Expanded([130, 7, 40], [200, 90, 61], heads=3)  # their keys share tiles of 128
        want = [x.copy() for x in e.run()]
        for t in (e.qd[130:137], e.kv[200:290], e.rd[200:290]):
            t.fill_(what)
        o, lse = e.run()
        assert int(e.err.item()) == 0 and np.isnan(o[130:137]).all()
        for rows in (slice(0, 130), slice(137, None)):
            assert np.array_equal(o[rows], want[0][rows]) and np.array_equal(lse[rows], want[1][rows])


@pytest.mark.parametrize("heads", [16, 128])
def test_two_graphs_share_a_workspace(heads):
    """Replayed in turn on one stream, with calls of the expanded form in the same workspace between them."""
    cases = [Case([1, 3], [4000, 700], heads=heads, seed=1), Case([2, 1], [90, 6000], heads=heads, seed=2)]
    e = Expanded([300, 1], [900, 3000], heads=2)
    want = [c.run()[0].copy() for c in cases]
    want_e = e.run()[0].copy()
    e.ws = cases[1].ws = cases[0].ws
    cases[1].args, e.args = cases[1].make_args(), e.make_args()
    s, graphs = torch.cuda.Stream(), []
    torch.cuda.synchronize()
    for c in cases:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            B.moe_attn_latent(c.cache, c.args)
        c.od.fill_(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(3):
            for g in graphs:
                g.replay()
            B.moe_attn_expanded(e.args)
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        assert np.array_equal(c.od[:sum(c.q_lens), :heads, :L].double().cpu().numpy(), w) and int(c.err.item()) == 0
    assert np.array_equal(e.od[:301, :2, :128].double().cpu().numpy(), want_e)
    assert int(e.ws[:4096].count_nonzero().item()) == 0
