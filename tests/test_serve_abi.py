"""Host-side checks of the serving operators (no GPU needed): what the C ABI and the binding
refuse before anything is enqueued, empty calls, and the plain implementations the GPU
tests compare with."""
import ctypes
import math

import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from serve_ref import attention, dequantise, e4m3_table, quantise, verify

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 4


class Pointers:
    """Distinct 16-byte aligned pointers (plus `off` bytes), 1 MB apart: with a GPU into one real
    zeroed buffer, so that a host check that ever let a call through would not run a kernel on
    a made-up address; without one, small integers (no kernel can launch)."""

    def __init__(self):
        self.t = torch.zeros(1 << 30, dtype=torch.uint8, device="cuda") if torch.cuda.is_available() else None
        self.next = (self.t.data_ptr() if self.t is not None else 0) + (1 << 20)

    def __call__(self, off=0):
        p = self.next + off
        self.next += 1 << 20
        assert self.t is None or self.next <= self.t.data_ptr() + self.t.numel()
        return p


@pytest.fixture
def P():
    return Pointers()


def cache(P, dtype=B.BF16, pages=4, page=16, heads=2, D=128, **kw):
    fp8 = dtype == B.FP8_E4M3
    f = dict(k=P(), v=P(), k_scale=P() if fp8 else None, v_scale=P() if fp8 else None, dtype=dtype, num_pages=pages,
             page_size=page, num_heads=heads, head_dim=D, stride_page=heads * page * D, stride_head=page * D,
             stride_token=D)
    f.update(kw)
    return B.MoeKvCache(**f)


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(num_pages=0), INVALID),
              (dict(num_heads=0), INVALID), (dict(page_size=-16), INVALID), (dict(dtype=B.F32), UNSUPPORTED),
              (dict(dtype=7), UNSUPPORTED), (dict(D=96), UNSUPPORTED), (dict(D=256), UNSUPPORTED),
              (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(stride_token=120), INVALID),
              (dict(stride_page=0), INVALID), (dict(stride_head=64), INVALID), (dict(stride_token=129), ALIGNMENT),
              (dict(stride_page=4100), ALIGNMENT), (dict(stride_page=1 << 39), UNSUPPORTED)]


@pytest.mark.parametrize("bad,want", BAD_CACHES)
def test_bad_caches(P, bad, want):
    L, c = B.lib(), cache(P, **bad)
    ref = ctypes.byref(c)
    assert L.moe_kv_write(ref, 1, P(), P(), 256, 256, 128, P(), None, 0, None) == want
    assert L.moe_kv_read(ref, 1, 1, P(), 1, P(), P(), P(), P(), None, 0, None) == want
    a = B.MoeAttnArgs()
    assert L.moe_attn_paged(ref, ctypes.byref(a), 0, None) == want
    assert L.moe_attn_workspace_size(ref, 8) == 0


def test_scales_go_with_the_type(P):
    L = B.lib()
    for c in (cache(P, k_scale=P()), cache(P, B.FP8_E4M3, v_scale=None)):
        assert L.moe_kv_write(ctypes.byref(c), 1, P(), P(), 256, 256, 128, P(), None, 0, None) == INVALID
    for f in ("k", "v", "k_scale"):
        c = cache(P, B.FP8_E4M3, **{f: P(8)})
        assert L.moe_kv_write(ctypes.byref(c), 1, P(), P(), 256, 256, 128, P(), None, 0, None) == ALIGNMENT
    c = cache(P, B.FP8_E4M3, stride_token=136)  # 8 bytes off
    assert L.moe_kv_write(ctypes.byref(c), 1, P(), P(), 256, 256, 128, P(), None, 0, None) == ALIGNMENT


def test_write_and_read_arguments(P):
    L, c = B.lib(), cache(P)
    ref = ctypes.byref(c)
    w = lambda T=1, k=1, v=1, lk=256, lv=256, hs=128, s=1, mis=0: L.moe_kv_write(
        ref, T, P(mis) if k else None, P() if v else None, lk, lv, hs, P() if s else None, None, 0, None)
    assert w(T=0, k=0, v=0, s=0) == 0
    assert w(T=-1) == w(k=0) == w(v=0) == w(s=0) == w(lk=-8) == w(hs=-8) == w(T=1 << 29) == INVALID
    assert w(mis=8) == w(lk=257) == w(lv=4) == w(hs=130) == ALIGNMENT
    r = lambda B_=1, T=1, t=1, ld=1, k=1, mis=0: L.moe_kv_read(
        ref, B_, T, P() if t else None, ld, P(), P(), P(mis) if k else None, P(), None, 0, None)
    assert r(B_=0) == r(T=0) == 0
    assert r(B_=-1) == r(T=-1) == r(t=0) == r(ld=-1) == r(k=0) == INVALID
    assert r(mis=4) == ALIGNMENT


def attn(P, c, **kw):
    f = dict(q=P(), o=P(), lse=None, q_ld=1024, q_head_stride=128, o_ld=1024, o_head_stride=128, cu_q=P(), kv_len=P(),
             block_table=P(), table_ld=4, T=1, B=1, max_q=1, max_kv=64, num_q_heads=8, scale=0.1, causal=1, window=0,
             err_flag=None, workspace=P(), workspace_bytes=1 << 20)
    f.update(kw)
    return B.lib().moe_attn_paged(ctypes.byref(c), ctypes.byref(B.MoeAttnArgs(**f)), 0, None)


def test_attention_arguments(P):
    c = cache(P)
    for kw in (dict(T=0, q=None), dict(B=0), dict(max_q=0)):
        assert attn(P, c, **kw) == 0
    for kw in (dict(T=-1), dict(B=-1), dict(max_q=-1), dict(max_kv=-1), dict(table_ld=-1), dict(window=-1),
               dict(num_q_heads=0), dict(num_q_heads=7), dict(scale=math.nan), dict(scale=math.inf), dict(causal=2),
               dict(q=None), dict(o=None), dict(cu_q=None), dict(kv_len=None), dict(block_table=None), dict(q_ld=-8),
               dict(o_head_stride=-8)):
        assert attn(P, c, **kw) == INVALID, kw
    big = 1 << 30
    for kw in (dict(num_q_heads=130), dict(B=8193), dict(T=big, max_kv=big), dict(T=big + 1), dict(max_kv=big + 1)):
        assert attn(P, c, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=P(8)), dict(o=P(2)), dict(q_ld=1028), dict(q_head_stride=12), dict(o_ld=4)):
        assert attn(P, c, **kw) == ALIGNMENT, kw
    assert attn(P, c, workspace=None) == attn(P, c, workspace_bytes=100) == WORKSPACE
    assert B.lib().moe_attn_paged(ctypes.byref(c), None, 0, None) == INVALID
    assert B.moe_attn_workspace_size(c, 8) > 0 and B.moe_attn_workspace_size(c, 7) == 0


def test_verify_arguments(P):
    L = B.lib()

    def v(B_=1, V=100, M=3, dt=B.F32, t=1, tl=100, d=1, dl=100, cu=1, ud=1, out=1, n=1, mis=0):
        return L.moe_draft_verify(B_, V, M, dt, P(mis) if t else None, tl, P() if d else None, dl, P() if cu else None,
                                  P(), P(), P() if ud else None, P() if out else None, P() if n else None, None, 0,
                                  None)

    assert v(B_=0) == 0
    assert v(B_=-1) == v(V=0) == v(M=-1) == v(tl=99) == v(dl=99) == v(t=0) == v(cu=0) == v(ud=0) == v(out=0) == \
        v(n=0) == INVALID
    assert v(dt=B.FP8_E4M3) == v(M=256) == UNSUPPORTED
    assert v(V=(1 << 23) + 1, tl=1 << 24, dl=1 << 24) == UNSUPPORTED
    assert v(mis=2) == ALIGNMENT


def test_verify_with_a_row_count(P):
    """moe_draft_verify_ex refuses a negative count, and otherwise what moe_draft_verify refuses."""
    v = lambda N=3, V=100: B.lib().moe_draft_verify_ex(1, N, V, 3, B.F32, P(), 100, P(), 100, P(), P(), P(), P(), P(), None,
                                                       None, 0, None)
    assert v(N=-1) == v(V=0) == v() == INVALID  # the last: no out_len


def test_the_binding_checks_tensors():
    z = torch.zeros
    bf, i32 = torch.bfloat16, torch.int32
    k = z(3, 2, 16, 64, dtype=bf)
    c = B.kv_cache(k, k)
    assert (c.num_pages, c.num_heads, c.page_size, c.head_dim, c.dtype) == (3, 2, 16, 64, B.BF16)
    t = z(3, 16, 2, 64, dtype=bf).transpose(1, 2)
    c2 = B.kv_cache(t, t)
    assert (c2.stride_page, c2.stride_head, c2.stride_token) == (2048, 64, 128)
    q8, s = k.to(torch.float8_e4m3fn), z(3, 2, 16, dtype=torch.uint8)
    assert B.kv_cache(q8, q8, s, s).dtype == B.FP8_E4M3
    for bad in ((k.float(), k.float()), (k, k[:2]), (k, t), (k, k, s, s), (q8, q8), (q8, q8, s, s[:2]),
                (k.transpose(2, 3), k.transpose(2, 3)), (k[0], k[0])):
        with pytest.raises(ValueError):
            B.kv_cache(*bad)
    x, slots = z(5, 2, 64, dtype=bf), z(5, dtype=torch.int64)
    for bad in ((x[:, :1], x, slots), (x.float(), x, slots), (x, x, slots[:4]), (x, x, slots.int())):
        with pytest.raises(ValueError):
            B.moe_kv_write(c, *bad)
    tab, st, cu = z(1, 4, dtype=i32), z(1, dtype=i32), z(2, dtype=i32)
    for bad in ((tab, st, cu, x, x[:4]), (tab.long(), st, cu, x, x), (tab, st, st, x, x)):
        with pytest.raises(ValueError):
            B.moe_kv_read(c, *bad)
    q = z(5, 4, 64, dtype=bf)
    for bad in ((q, q[:, :2], cu, st, tab), (q, q, st, st, tab), (q, q, cu, st, tab[0]), (q.float(), q, cu, st, tab)):
        with pytest.raises(ValueError):
            B.attn_args(*bad, 5, 64, 0.1)
    with pytest.raises(ValueError):
        B.attn_args(q, q, cu, st, tab, 5, 64, 0.1, lse=z(4, 5))
    with pytest.raises(B.MoeError) as e:
        B.moe_attn_paged(c, B.attn_args(q, q, cu, st, tab, 5, 64, 0.1), stream=0)
    assert e.value.status == WORKSPACE
    p, f = z(3, 50), z(2)
    out = z(1, 3, dtype=i32)
    ids = z(2, dtype=i32)
    ok = (p, z(2, 50), cu, ids, f, z(1), out, st)
    for i, bad in ((0, p.double()), (0, p[:2]), (1, z(2, 49)), (1, z(2, 50, dtype=bf)), (2, st), (3, ids.long()),
                   (4, z(3)), (6, out.long()), (6, z(2, 3, dtype=i32))):
        args = list(ok)
        args[i] = bad
        with pytest.raises(ValueError):
            B.moe_draft_verify(*args)


def test_rows_of_o_lie_apart(P):
    """Overlapping rows of o are refused, whatever their order; layouts without overlap are not (they go on to
    the check of the workspace)."""
    c = cache(P)  # heads of 128
    for o_ld, o_head in ((0, 128), (1024, 0), (1024, 64), (120, 128), (128, 128), (896, 128), (128, 512), (128, 632),
                         (128 * 5, 128 * 3), (256, 384)):
        assert attn(P, c, T=5, max_q=5, o_ld=o_ld, o_head_stride=o_head, workspace=None) == INVALID, (o_ld, o_head)
    for o_ld, o_head in ((1024, 128), (128, 640), (128, 648), (2048, 256), (1 << 30, 128), (128 * 8, 128 * 40), (256, 128 * 11)):
        assert attn(P, c, T=5, max_q=5, o_ld=o_ld, o_head_stride=o_head, workspace=None) == WORKSPACE, (o_ld, o_head)
    # by counting, for every small layout of both orders
    at0 = P()
    for T in (1, 2, 3):
        for ld in range(0, 1200, 64):
            for hs in range(0, 1200, 64):
                at = sorted(t * ld + h * hs for t in range(T) for h in range(4))
                apart = all(b - a >= 128 for a, b in zip(at, at[1:]))
                got = attn(lambda: at0, c, T=T, max_q=T, num_q_heads=4, o_ld=ld, o_head_stride=hs, workspace=None)
                assert got == (WORKSPACE if apart else INVALID), (T, ld, hs)
    assert attn(P, c, o_ld=0, workspace=None) == WORKSPACE, "one token: its stride is not used"
    big = 1 << 39
    for kw in (dict(o_ld=big), dict(q_ld=big), dict(o_head_stride=big), dict(q_head_stride=big)):
        assert attn(P, c, T=2, max_q=2, workspace=None, **kw) == UNSUPPORTED, kw


@pytest.mark.parametrize("D,other", [(64, 128), (128, 64)])
def test_the_binding_checks_the_width_of_q_and_o(D, other):
    """Heads of another width than the cache's are refused before the C call, which sees pointers and
    strides only: too narrow ones would be read and written past their end."""
    z, bf, i32 = torch.zeros, torch.bfloat16, torch.int32
    k = z(3, 2, 16, D, dtype=bf)
    c = B.kv_cache(k, k)
    tab, kv, cu = z(1, 4, dtype=i32), z(1, dtype=i32), z(2, dtype=i32)
    q = z(5, 4, other, dtype=bf)
    with pytest.raises(ValueError):
        B.moe_attn_paged(c, B.attn_args(q, q.clone(), cu, kv, tab, 5, 64, 0.1), stream=0)


# ---------------------------------------------------------------- the plain implementations
def test_reference_quantisation():
    t = e4m3_table()
    assert np.array_equal(t, torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    rng = np.random.default_rng(0)
    x = torch.tensor(rng.standard_normal((50, 64)) * np.exp(rng.uniform(-20, 20, (50, 1)))).to(torch.bfloat16)
    codes, s = quantise(x.double().numpy())
    e = s.astype(np.int64) - 127
    amax = x.double().abs().amax(-1).numpy()
    assert (amax <= 448 * 2.0**e).all() and (amax > 448 * 2.0**(e - 1)).all()
    want = (x.double() * torch.tensor(2.0**-e)[:, None]).float().to(torch.float8_e4m3fn)
    assert np.array_equal(codes, want.view(torch.uint8).numpy())
    assert np.array_equal(dequantise(codes, s), (want.double() * torch.tensor(2.0**e)[:, None]).numpy())


def test_reference_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((3, 4, 8)), rng.standard_normal((9, 2, 8)), rng.standard_normal((9, 2, 8))
    o, lse, _ = attention(q, k, v, 9, 0.5)
    s = np.einsum("ihd,jhd->hij", q, k.repeat(2, 1)) * 0.5
    s[:, np.arange(9)[None] > np.arange(6, 9)[:, None]] = -np.inf
    p = np.exp(s)
    assert np.allclose(o, np.einsum("hij,jhd->ihd", p / p.sum(-1, keepdims=True), v.repeat(2, 1)))
    assert np.allclose(lse, np.log(p.sum(-1)).T)
    o, lse, _ = attention(q, k[:2], v[:2], 2, 0.5)
    assert np.isneginf(lse[0]).all() and (o[0] == 0).all()
    assert np.allclose(o[1], v[:1].repeat(2, 1))


def test_reference_verify():
    t = np.array([[.5, .5, 0, 0], [0, 0, .25, .75], [1, 0, 0, 0]], np.float32)
    d = np.array([[.25, .75, 0, 0], [0, 0, .5, .5]], np.float32)
    # the first is kept below 0.5 / 0.75; the second (token 2) below 0.25 / 0.5, then 3 has the rest
    out, n = verify(t, d, [0, 2], [1, 2], [0.6, 0.6], [0.9], 2)
    assert out.tolist() == [[1, 3, -1]] and n.tolist() == [2]
    out, n = verify(t, d, [0, 2], [1, 2], [0.7, 0.0], [0.9], 2)
    assert out.tolist() == [[0, -1, -1]] and n.tolist() == [1]
    out, n = verify(t, d, [0, 2], [1, 2], [0.0, 0.0], [0.9], 2)
    assert out.tolist() == [[1, 2, 0]] and n.tolist() == [3]
