"""Draft verification on the GPU against exact whole-number arithmetic in Python."""
import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from serve_ref import verify

pytestmark = pytest.mark.gpu
DEV = "cuda"


def run(target, draft, lens, ids, u, u_draw, max_draft, pad=0, dtype=torch.float32, **kw):
    def rows(x):
        if x is None:
            return None
        t = torch.full((x.shape[0], x.shape[1] + pad), 3.0, dtype=dtype, device=DEV)
        t[:, :x.shape[1]] = torch.tensor(x, device=DEV).to(dtype)
        return t[:, :x.shape[1]]

    t, d = rows(target), rows(draft)
    n = len(lens)
    out = torch.full((n, max_draft + 1), 55, dtype=torch.int32, device=DEV)
    length = torch.full((n,), 55, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    cu = np.cumsum([0] + lens)
    dev = lambda a, ty: torch.tensor(np.asarray(a), dtype=ty, device=DEV)
    B.moe_draft_verify(t, d, dev(cu, torch.int32), dev(ids, torch.int32), dev(u, torch.float32),
                       dev(u_draw, torch.float32), out, length, err_flag=err, **kw)
    torch.cuda.synchronize()
    host = lambda x: None if x is None else x.float().cpu().numpy()
    want, wl = verify(host(t), host(d), cu, ids, np.float32(u), np.float32(u_draw), max_draft)
    assert np.array_equal(length.cpu().numpy(), wl)
    assert np.array_equal(out.cpu().numpy(), want)
    return out.cpu().numpy(), length.cpu().numpy(), int(err.item())


def softmax(x):
    e = np.exp(x - x.max(-1, keepdims=True))
    return (e / e.sum(-1, keepdims=True)).astype(np.float32)


def batch(lens, V, seed, near=0.7):
    rng = np.random.default_rng(seed)
    N, n = sum(lens), len(lens)
    z = rng.standard_normal((N + n, V)) * 2.5
    cu = np.cumsum([0] + lens)
    row = np.array([cu[b] + b + i for b in range(n) for i in range(lens[b])], dtype=np.int64)
    draft = softmax(z[row] + rng.standard_normal((N, V)) * near) if N else np.zeros((0, V), np.float32)
    ids = [int(rng.choice(V, p=d.astype(np.float64) / d.sum(dtype=np.float64))) for d in draft]
    return softmax(z), draft, ids, rng.random(N, dtype=np.float32), rng.random(n, dtype=np.float32)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 3, 127, 128, 129, 1000, 4099, 32001, 50000])
@pytest.mark.parametrize("lens", [[4], [0, 1, 5, 3, 0, 2]])
def test_against_exact(dtype, V, lens):
    for seed in range(3):
        t, d, ids, u, ud = batch(lens, V, seed)
        _, _, err = run(t, d, lens, ids, u, ud, 5, dtype=dtype)
        assert err == 0


@pytest.mark.parametrize("pad", [0, 1, 3, 4])
def test_row_strides(pad):
    lens = [3, 0, 2]
    t, d, ids, u, ud = batch(lens, 1024, 9)
    run(t, d, lens, ids, u, ud, 3, pad=pad)


def test_every_length_and_more_requests_than_clusters():
    lens = [i % 40 for i in range(120)]
    t, d, ids, u, ud = batch(lens, 300, 4, near=0.05)  # most tokens are kept: past 32
    for kw in ({}, dict(max_ctas=8), dict(max_ctas=1)):
        out, n, _ = run(t, d, lens, ids, u, ud, 64, **kw)
    assert n.max() > 33


def test_no_drafts_at_all():
    t, d, ids, u, ud = batch([0, 0, 0], 777, 1)
    run(t, None, [0, 0, 0], ids, u, ud, 4)
    run(t, d, [0, 0, 0], ids, u, ud, 0)


def test_deterministic_draft():
    lens = [4, 2, 0, 3]
    t, _, ids, u, ud = batch(lens, 500, 2)
    for scale in (1.0, 0.02):
        run(t, None, lens, ids, u * np.float32(scale), ud, 4)


def test_extreme_numbers():
    """u at 0 and just below 1 and outside; mass at the first and at the last token only."""
    V = 1000
    for where in (0, 1, 511, 998, 999):
        t = np.zeros((3, V), np.float32)
        t[:, where] = 1.0
        d = np.full((2, V), 1.0 / V, np.float32)
        for u in (0.0, 1 - 2.0**-24, 1.5, -1.0):
            run(t, d, [2], [where, (where + 1) % V], [u, u], [u], 2)
    # the largest sums there can be, and the smallest nonzero ones
    t = np.ones((1, 5000), np.float32)
    run(t, None, [0], [], [], [1 - 2.0**-24], 0)
    t = np.full((1, 5000), 2.0**-40, np.float32)
    run(t, None, [0], [], [], [0.77], 0)


def test_no_mass_left():
    """A refused token where the target has nothing beyond the draft: drawn from the target; where
    that has nothing either: -1 and an error."""
    V = 300
    p = softmax(np.random.default_rng(0).standard_normal((2, V)))
    d = p[:1].copy()
    out, n, err = run(p, d, [1], [5], [1 - 2.0**-24], [0.4], 1)
    d = np.maximum(p[:1], 0.5).astype(np.float32)  # above the target everywhere
    out, n, err = run(p, d, [1], [5], [0.9], [0.4], 1)
    assert err == 0 and n[0] == 1 and out[0, 0] >= 0
    for bad in (0.0, float("nan")):
        out, n, err = run(np.full((2, V), bad, np.float32), d, [1], [5], [0.9], [0.4], 1)
        assert err == 7 and out[0].tolist() == [-1, -1] and n[0] == 1


def test_ids_out_of_range():
    lens = [3, 2]
    t, d, ids, u, ud = batch(lens, 400, 3)
    for bad in (-1, 400, 2**31 - 1):
        ids2 = list(ids)
        ids2[0] = bad
        _, n, err = run(t, d, lens, ids2, u, ud, 3)
        assert err == 7 and n[0] == 1


def test_too_many_drafts_for_a_row():
    t, d, ids, u, ud = batch([3, 1], 100, 3)
    out = torch.full((2, 3), 55, dtype=torch.int32, device=DEV)
    n = torch.full((2,), 55, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    dev = lambda a, ty: torch.tensor(np.asarray(a), dtype=ty, device=DEV)
    f = torch.float32
    B.moe_draft_verify(dev(t, f), dev(d, f), dev([0, 3, 4], torch.int32), dev(ids, torch.int32), dev(u, f), dev(ud, f),
                       out, n, err_flag=err)
    assert int(err.item()) == 7 and n[0].item() == 0 and out[0].tolist() == [-1, -1, -1] and n[1].item() in (1, 2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_past_the_inputs_are_not_read(dtype):
    """cu_draft beyond the rows that there are (here: parts of larger buffers): those requests are refused, the
    others are not touched by it."""
    lens = [2, 1, 3, 1]
    t, d, ids, u, ud = batch(lens, 200, 5)
    dev = lambda a, ty: torch.tensor(np.asarray(a), dtype=ty, device=DEV)
    f = torch.float32
    full = dev(t, dtype), dev(d, dtype), dev(ids, torch.int32), dev(u, f), dev(ud, f)
    cut = lambda n: (full[0][:n + 4], full[1][:n], full[2][:n], full[3][:n], full[4])

    def call(n, cu):
        out = torch.full((4, 4), 55, dtype=torch.int32, device=DEV)
        length = torch.full((4,), 55, dtype=torch.int32, device=DEV)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        a = cut(n)
        B.moe_draft_verify(a[0], a[1], dev(cu, torch.int32), a[2], a[3], a[4], out, length, err_flag=err)
        return out.tolist(), length.tolist(), int(err.item())

    out, length, err = call(7, [0, 2, 3, 6, 7])
    assert err == 0 and min(length) >= 1
    for n, refused in ((6, [3]), (5, [2, 3]), (2, [1, 2, 3])):
        o, ln, e = call(n, [0, 2, 3, 6, 7])
        assert e == 7
        for b in range(4):
            if b in refused:
                assert ln[b] == 0 and o[b] == [-1] * 4
            else:
                assert (o[b], ln[b]) == (out[b], length[b])
    # a descending one, and one that starts past the end
    _, ln, e = call(7, [0, 9, 3, 6, 7])
    assert e == 7 and ln[:2] == [0, 0] and ln[2:] == length[2:]
    _, ln, e = call(7, [0, 2, 2**31 - 1, 2**31 - 1, -2**31])
    assert e == 7 and ln[0] == length[0] and ln[1:] == [0, 0, 0]


def test_every_number_of_the_draw():
    """All 2^24 values of u_draw over one distribution of 300 tokens: how often a token comes is its
    probability times 2^24, within one: those smaller than 2^-24 come once or never."""
    V, n = 300, 1 << 24
    p = softmax(np.random.default_rng(5).standard_normal((1, V)) * 6).astype(np.float32)
    assert (p < 2.0**-24).sum() > 20
    step = 1 << 20
    t = torch.tensor(p, device=DEV).repeat(step, 1)
    got = torch.zeros(V, dtype=torch.int64, device=DEV)
    out = torch.empty(step, 1, dtype=torch.int32, device=DEV)
    length = torch.empty(step, dtype=torch.int32, device=DEV)
    cu = torch.zeros(step + 1, dtype=torch.int32, device=DEV)
    for a in range(0, n, step):
        u = torch.arange(a, a + step, device=DEV).float() * 2.0**-24
        B.moe_draft_verify(t, None, cu, None, None, u, out, length)
        got += torch.bincount(out[:, 0].long(), minlength=V)
    w = np.floor(p[0].astype(np.float64) * 2.0**40)
    assert np.abs(got.cpu().numpy() - w / w.sum() * n).max() < 1.0


def test_distribution():
    """Kept and drawn tokens together follow the target: 40000 trials over 12 tokens, a chi-squared
    statistic of 11 degrees below 45 (probability of more: 5e-6)."""
    rng = np.random.default_rng(11)
    V, n = 12, 40000
    z = rng.standard_normal((1, V)) * 1.5
    p, q = softmax(z), softmax(z + rng.standard_normal((1, V)))
    ids = rng.choice(V, size=n, p=q[0].astype(np.float64) / q[0].sum(dtype=np.float64))
    f = lambda a: torch.tensor(a, dtype=torch.float32, device=DEV)
    out = torch.empty(n, 2, dtype=torch.int32, device=DEV)
    length = torch.empty(n, dtype=torch.int32, device=DEV)
    B.moe_draft_verify(f(p).repeat(2 * n, 1), f(q).repeat(n, 1), torch.arange(n + 1, dtype=torch.int32, device=DEV),
                       torch.tensor(ids, dtype=torch.int32, device=DEV), f(rng.random(n)), f(rng.random(n)), out,
                       length)
    got = np.bincount(out[:, 0].cpu().numpy(), minlength=V)
    want = p[0].astype(np.float64) * n
    assert ((got - want)**2 / want).sum() < 45


def test_graph():
    lens = [4, 2, 0, 3]
    t, d, ids, u, ud = batch(lens, 5000, 2)
    dev = lambda a, ty: torch.tensor(np.asarray(a), dtype=ty, device=DEV)
    f = torch.float32
    args = [dev(t, f), dev(d, f), dev(np.cumsum([0] + lens), torch.int32), dev(ids, torch.int32), dev(u, f), dev(ud, f)]
    out = torch.empty(4, 5, dtype=torch.int32, device=DEV)
    n = torch.empty(4, dtype=torch.int32, device=DEV)
    B.moe_draft_verify(*args, out, n)
    want, wl = out.clone(), n.clone()
    g = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=s):
        B.moe_draft_verify(*args, out, n)
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(n, wl)
