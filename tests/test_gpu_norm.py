"""moe_block_norm and moe_latent_write on the GPU against plain implementations in 64 bits."""
import numpy as np
import pytest
import torch

from latent_ref import U_BF16, U_F32, block_norm, rms
from moe_expert_dispatch_route_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {torch.float32: U_F32, torch.bfloat16: U_BF16}


def near(got, want, extra, what):
    """One rounding to the type of `got`, and `extra`, what fp32's arithmetic before it may be off by."""
    bound = HALF[got.dtype] * np.abs(want) + extra + 1e-30
    off = np.abs(got.double().cpu().numpy() - want)
    assert np.all(off <= bound), f"{what}: {(off > bound).sum()} of {off.size} off, worst {(off / bound).max():.3f} bounds"


def run(T, H, dtype="bf16", resid="bf16", post=False, gate=0, keep=True, normed=True, scale=0.75, eps=1e-6, seed=0,
        inplace=False, std=1.0, max_ctas=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s, t=dtype: torch.randn(*s, generator=g, device=DEV).to(TYPES[t])
    y, r = (rand(T, H) * std).to(TYPES[dtype]), rand(T, H, t=resid) if resid else None
    pre, w = rand(H), rand(H) if post else None
    gt = rand(1 if gate == 1 else T, H) if gate else None
    d = lambda t: None if t is None else t.double().cpu().numpy()
    R, out = block_norm(d(y), d(pre) if normed else None, d(r), d(w), d(gt), scale, eps)
    X = block_norm(d(y), None, None, d(w), d(gt), scale, eps)[0]
    ro = (r if inplace and r is not None else torch.full_like(y, 7, dtype=TYPES[resid or dtype])) if keep else None
    o = (y if inplace else torch.full_like(y, 7)) if normed else None
    B.moe_block_norm(y, o, pre if normed else None, resid=r, resid_out=ro, post_weight=w, gate=gt, scale=scale, eps=eps,
                     max_ctas=max_ctas)
    torch.cuda.synchronize()
    # a sum of H squares in fp32 is off by (H / 256 + 10) half steps at most (threads' sums, then a tree), its root
    # by half of that, and a handful of products by one each; x's part of r' carries the first norm's
    e = (H / 256 + 32) * U_F32
    if keep:
        near(ro, R, e * np.abs(X) + 2 * U_F32 * np.abs(R), "resid_out")
    if normed:
        # the second norm: r' is off by e |x|; its root mean square by at most e times that of x over that of r'
        ratio = np.sqrt((X * X).mean(-1, keepdims=True) / ((R * R).mean(-1, keepdims=True) + eps))
        near(o, out, np.abs(out) * e * (1 + ratio) + e * np.abs(X) * np.abs(d(pre)) /
             np.sqrt((R * R).mean(-1, keepdims=True) + eps), "out")


@pytest.mark.parametrize("H", [8, 72, 256, 264, 512, 1000, 2048, 2056, 4096, 7168, 8200, 16384])
@pytest.mark.parametrize("dtype,resid", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
def test_widths_and_types(H, dtype, resid):
    run(5, H, dtype, resid, post=True, gate=2, seed=H)
    run(3, H, dtype, resid, seed=H + 1)


@pytest.mark.parametrize("T", [1, 2, 7, 8, 9, 700])
@pytest.mark.parametrize("gate", [0, 1, 2])
def test_tokens_and_gates(T, gate):
    run(T, 392, post=True, gate=gate, seed=T)
    run(T, 136, gate=gate, seed=T, max_ctas=1)
    run(T, 2048, post=True, gate=gate, seed=T, max_ctas=3)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("resid", [None, "bf16", "f32"])
@pytest.mark.parametrize("keep,normed", [(True, False), (False, True), (True, True)])
def test_parts_left_out(post, resid, keep, normed):
    run(300, 1544, resid=resid, post=post, keep=keep, normed=normed, scale=-1.5)
    run(300, 640, "f32", resid=resid, post=post, keep=keep, normed=normed, max_ctas=2)


def test_in_place_and_ranges():
    run(65, 7168, post=True, gate=1, inplace=True)
    run(65, 1024, "f32", "f32", inplace=True)
    run(9, 512, std=1e-12, post=True, eps=1e-30)  # eps matters next to 1e-24
    run(9, 512, "f32", "f32", std=1e15, post=True)


@pytest.mark.parametrize("dtype,resid", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("H", [768, 1024, 1032, 2048, 2056, 4104, 6152, 8192, 16384])
def test_rows_in_turn(H, dtype, resid):
    """More rows than a CTA's ring holds, several times over, in place too, and one norm of the two."""
    run(29, H, dtype, resid, post=True, gate=2, seed=H, max_ctas=2)
    run(29, H, dtype, resid, post=True, gate=1, seed=H + 1, max_ctas=1, inplace=True)
    run(29, H, dtype, resid, seed=H + 2, max_ctas=2, inplace=True)
    run(29, H, dtype, resid, post=True, normed=False, seed=H + 3, max_ctas=1)
    run(29, H, dtype, None, keep=False, seed=H + 4, max_ctas=1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H", [256, 520, 1024, 2048, 2304, 4096, 5000, 7168, 16384])
def test_a_row_does_not_depend_on_the_others(H, dtype):
    T = 5003 if H <= 1024 else 701
    y, r = torch.randn(T, H, device=DEV).to(TYPES[dtype]), torch.randn(T, H, device=DEV)
    w, gate = torch.randn(H, device=DEV).to(TYPES[dtype]), torch.randn(T, H, device=DEV).to(TYPES[dtype])
    out, ro = torch.empty_like(y), torch.empty_like(r)
    B.moe_block_norm(y, out, w, resid=r, resid_out=ro, post_weight=w, gate=gate)
    for t in (0, 333, T - 3):
        some = slice(t, t + 3)
        o, q = torch.empty_like(y[some]), torch.empty_like(r[some])
        B.moe_block_norm(y[some], o, w, resid=r[some], resid_out=q, post_weight=w, gate=gate[some])
        assert torch.equal(o, out[some]) and torch.equal(q, ro[some])


def test_many_tokens_and_rows_behind_them():
    T, H = 40001, 256
    y = torch.randn(T, H, device=DEV).to(torch.bfloat16)
    out = torch.full((T + 3, H), 7.0, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(H, dtype=torch.bfloat16, device=DEV)
    B.moe_block_norm(y, out[:T], w)
    assert torch.all(out[T:] == 7.0)
    want = rms(y.double().cpu().numpy(), 1.0, 1e-6)
    near(out[:T], want, 40 * U_F32 * np.abs(want), "out")


@pytest.mark.parametrize("H", [1024, 8192])
def test_offsets_past_31_bits(H):
    T = (1 << 31) // H + 300
    y, w = torch.full((T, H), 0.5, dtype=torch.bfloat16, device=DEV), torch.ones(H, dtype=torch.bfloat16, device=DEV)
    tail = torch.randn(300, H, device=DEV).to(torch.bfloat16)
    y[-300:] = tail
    B.moe_block_norm(y, y, w)
    out = torch.empty_like(tail)
    B.moe_block_norm(tail, out, w)
    assert torch.equal(y[-300:], out) and torch.all(y[:-300] == 1.0)


def test_a_row_of_zeros():
    y, w = torch.zeros(3, 2048, dtype=torch.bfloat16, device=DEV), torch.ones(2048, dtype=torch.bfloat16, device=DEV)
    y[1] = 1.0
    out = torch.empty_like(y)
    B.moe_block_norm(y, out, w, eps=1e-6)
    assert torch.all(out[[0, 2]] == 0.0) and torch.all(out[1] == 1.0)
    B.moe_block_norm(y, out, w, eps=0.0)
    assert torch.all(out[[0, 2]].isnan()) and torch.all(out[1] == 1.0)


def test_stream_and_graph():
    y, r = torch.randn(64, 2048, device=DEV).to(torch.bfloat16), torch.randn(64, 2048, device=DEV)
    w, out, ro = torch.ones(2048, dtype=torch.bfloat16, device=DEV), torch.empty_like(y), torch.empty_like(r)
    call = lambda: B.moe_block_norm(y, out, w, resid=r, resid_out=ro)
    call()
    want = (out.clone(), ro.clone())
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=s):
        call()
    out.zero_(), ro.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(ro, want[1])


# ------------------------------------------------------------------------------ latent cache
@pytest.mark.parametrize("T", [1, 3, 64, 1000])
@pytest.mark.parametrize("page,spare", [(16, 0), (64, 64), (128, 8)])
@pytest.mark.parametrize("norm", [False, True])
def test_latent_write(T, page, spare, norm):
    g = torch.Generator(device=DEV).manual_seed(T * page)
    pages = -(-T // page) + 2
    wide = torch.full((pages, page, 576 + spare), 3.0, dtype=torch.bfloat16, device=DEV)
    cache = B.latent_cache(wide[:, :, :576])
    down = torch.randn(T, 640, generator=g, device=DEV).to(torch.bfloat16)
    down[0] *= 1e-18  # a row beside which eps counts
    c, rope = down[:, 64:576], down[:, 576:]
    w = torch.randn(512, generator=g, device=DEV).to(torch.bfloat16) if norm else None
    slots = torch.randperm(pages * page, generator=g, device=DEV)[:T].contiguous()
    skip = slots.clone()
    skip[T // 2] = -5  # padding
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_latent_write(cache, c, rope, skip if T > 1 else slots, weight=w, eps=1e-6, err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    flat = wide.view(-1, 576 + spare)
    kept = torch.ones(T, dtype=torch.bool, device=DEV)
    if T > 1:
        kept[T // 2] = False
    at = slots[kept]
    assert torch.equal(flat[at, 512:576], rope[kept])
    if norm:
        want = rms(c[kept].double().cpu().numpy(), w.double().cpu().numpy(), 1e-6)
        near(flat[at, :512], want, 40 * U_F32 * np.abs(want), "latent vectors")
    else:
        assert torch.equal(flat[at, :512], c[kept])
    assert torch.all(flat[:, 576:] == 3.0)
    rest = torch.ones(pages * page, dtype=torch.bool, device=DEV)
    rest[at] = False
    assert torch.all(flat[rest] == 3.0), "other slots are left as they were"


def test_latent_write_past_the_pool():
    pool = torch.zeros(2, 16, 576, dtype=torch.bfloat16, device=DEV)
    x = torch.ones(3, 576, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_latent_write(B.latent_cache(pool), x[:, :512], x[:, 512:], torch.tensor([32, 31, 1 << 40], device=DEV),
                       err_flag=err, max_ctas=1)
    torch.cuda.synchronize()
    assert int(err.item()) == 7
    assert torch.all(pool.view(32, 576)[31] == 1) and torch.all(pool.view(32, 576)[:31] == 0)


def test_latent_write_other_orders():
    """A pool kept token first, and rows of c that one token's projection shares."""
    pool = torch.zeros(32, 4, 576, dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    x = torch.randn(1, 576, device=DEV).to(torch.bfloat16).expand(5, 576)
    slots = torch.tensor([0, 33, 66, 99, 127], device=DEV)
    B.moe_latent_write(B.latent_cache(pool), x[:, :512], x[:, 512:], slots)
    torch.cuda.synchronize()
    for s in slots.tolist():
        assert torch.equal(pool[s // 32, s % 32], x[0])
    assert int((pool != 0).any(-1).sum()) == 5
