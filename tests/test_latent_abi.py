"""Host-side checks of latent attention, tree attention and the norms around a block (no GPU needed): what the C
ABI and the binding refuse before anything is enqueued, empty calls, and the plain forms the GPU tests use."""
import ctypes
import math

import numpy as np
import pytest
import torch

import latent_ref as R
from moe_expert_dispatch_route_gb300 import binding as B
from test_serve_abi import ALIGNMENT, INVALID, UNSUPPORTED, WORKSPACE, P, cache  # noqa: F401

BIG = 1 << 30


def latent(P, pages=4, page=16, **kw):
    f = dict(kv=P(), dtype=B.BF16, num_pages=pages, page_size=page, latent=512, rope=64, stride_page=page * 576,
             stride_token=576)
    f.update(kw)
    return B.MoeLatentCache(**f)


@pytest.mark.parametrize("bad,want", [
    (dict(kv=None), INVALID), (dict(num_pages=0), INVALID), (dict(page_size=-16), INVALID), (dict(latent=0), INVALID),
    (dict(rope=-64), INVALID), (dict(stride_token=568), INVALID), (dict(stride_page=0), INVALID),
    (dict(dtype=B.F32), UNSUPPORTED), (dict(dtype=B.FP8_E4M3), UNSUPPORTED), (dict(latent=256), UNSUPPORTED),
    (dict(rope=128), UNSUPPORTED), (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED),
    (dict(stride_page=1 << 39), UNSUPPORTED), (dict(stride_token=580), ALIGNMENT), (dict(stride_page=9220), ALIGNMENT)])
def test_bad_latent_caches(P, bad, want):
    L, c = B.lib(), latent(P, **bad)
    ref = ctypes.byref(c)
    assert L.moe_latent_write(ref, 1, P(), 576, P(), 576, None, 1e-6, P(), None, 0, None) == want
    assert L.moe_attn_latent(ref, ctypes.byref(B.MoeAttnArgs()), None, 0, None) == want
    assert L.moe_attn_latent_workspace_size(ref, 16) == 0


def test_latent_write_arguments(P):
    L, c = B.lib(), latent(P)
    assert L.moe_latent_write(None, 1, P(), 576, P(), 576, None, 1e-6, P(), None, 0, None) == INVALID
    w = lambda T=1, x=1, r=1, s=1, lc=576, lr=576, eps=1e-6, off=(0, 0, 0): L.moe_latent_write(
        ctypes.byref(c), T, P(off[0]) if x else None, lc, P(off[1]) if r else None, lr, P(off[2]), eps,
        P() if s else None, None, 0, None)
    assert w(T=0, x=0, r=0, s=0) == 0
    assert w(T=-1) == w(x=0) == w(r=0) == w(s=0) == w(lc=-8) == w(lr=-8) == w(eps=-1.0) == w(eps=math.nan) == INVALID
    assert w(eps=math.inf) == INVALID
    assert w(off=(8, 0, 0)) == w(off=(0, 8, 0)) == w(off=(0, 0, 8)) == w(lc=580) == w(lr=4) == ALIGNMENT
    assert w(T=2, lc=1 << 39) == w(T=2, lr=1 << 39) == UNSUPPORTED
    c2 = latent(P, kv=P(8))
    assert L.moe_latent_write(ctypes.byref(c2), 1, P(), 576, P(), 576, None, 1e-6, P(), None, 0, None) == ALIGNMENT


def attn(P, tree=False, off=0, c=None, **kw):
    f = dict(q=P(), o=P(), lse=None, q_ld=16 * 576, q_head_stride=576, o_ld=16 * 512, o_head_stride=512, cu_q=P(),
             kv_len=P(), block_table=P(), table_ld=4, T=1, B=1, max_q=1, max_kv=64, num_q_heads=16, scale=0.1, causal=1,
             window=0, err_flag=None, workspace=P(), workspace_bytes=1 << 20)
    f.update(kw)
    return B.lib().moe_attn_latent(ctypes.byref(c or latent(P)), ctypes.byref(B.MoeAttnArgs(**f)),
                                   P(off) if tree else None, 0, None)


def test_latent_attention_arguments(P):
    for kw in (dict(T=0, q=None), dict(B=0), dict(max_q=0), dict(T=0, tree=True)):
        assert attn(P, **kw) == 0
    for kw in (dict(T=-1), dict(B=-1), dict(max_q=-1), dict(max_kv=-1), dict(table_ld=-1), dict(window=-1),
               dict(num_q_heads=0), dict(scale=math.nan), dict(scale=-0.5), dict(scale=math.inf), dict(causal=2),
               dict(q=None), dict(o=None), dict(cu_q=None), dict(kv_len=None), dict(block_table=None), dict(q_ld=-8),
               dict(o_head_stride=-8), dict(T=2, o_ld=504), dict(o_head_stride=504), dict(tree=True, causal=0),
               dict(tree=True, window=5), dict(T=3, o_ld=512, o_head_stride=512)):
        assert attn(P, **kw) == INVALID, kw
    for kw in (dict(num_q_heads=129), dict(B=8193), dict(T=BIG, max_kv=BIG), dict(T=BIG + 1), dict(max_kv=BIG + 1),
               dict(tree=True, max_q=65), dict(T=2, q_ld=1 << 39), dict(q_head_stride=1 << 39)):
        assert attn(P, **kw) == UNSUPPORTED, kw
    for kw in (dict(q=P(8)), dict(o=P(2)), dict(q_ld=9220), dict(q_head_stride=580), dict(o_ld=8196),
               dict(o_head_stride=516), dict(tree=True, off=4)):
        assert attn(P, **kw) == ALIGNMENT, kw
    assert attn(P, workspace=None) == attn(P, workspace_bytes=100) == WORKSPACE
    c = latent(P)
    assert B.lib().moe_attn_latent(ctypes.byref(c), None, None, 0, None) == INVALID
    assert B.moe_attn_latent_workspace_size(c, 128) > 0
    assert B.moe_attn_latent_workspace_size(c, 129) == B.moe_attn_latent_workspace_size(c, 0) == 0


def test_tree_arguments(P):
    c = cache(P)

    def call(tree=True, off=0, **kw):
        f = dict(q=P(), o=P(), lse=None, q_ld=1024, q_head_stride=128, o_ld=1024, o_head_stride=128, cu_q=P(), kv_len=P(),
                 block_table=P(), table_ld=4, T=1, B=1, max_q=1, max_kv=64, num_q_heads=8, scale=0.1, causal=1, window=0,
                 err_flag=None, workspace=P(), workspace_bytes=1 << 20)
        f.update(kw)
        return B.lib().moe_attn_tree(ctypes.byref(c), ctypes.byref(B.MoeAttnArgs(**f)), P(off) if tree else None, 0, None)

    assert call(T=0, tree=False) == call(B=0) == call(max_q=0) == 0
    assert call(tree=False) == call(causal=0) == call(window=3) == call(T=-1) == call(q=None) == call(num_q_heads=7) == INVALID
    assert call(max_q=65) == UNSUPPORTED and call(off=4) == ALIGNMENT
    assert call(workspace=None) == call(max_q=64, workspace_bytes=1) == WORKSPACE
    assert B.lib().moe_attn_tree(ctypes.byref(c), None, P(), 0, None) == INVALID
    bad = cache(P, D=96)
    assert B.lib().moe_attn_tree(ctypes.byref(bad), ctypes.byref(B.MoeAttnArgs(causal=1)), P(), 0, None) == UNSUPPORTED


def test_expanded_arguments(P):
    def call(**kw):
        f = dict(q=P(), k=P(), k_rope=P(), v=P(), o=P(), lse=None, q_ld=384, q_head_stride=192, k_ld=256, k_head_stride=128,
                 rope_ld=64, v_ld=256, v_head_stride=128, o_ld=256, o_head_stride=128, cu_q=P(), cu_kv=P(), T=2, S=2, B=1,
                 max_q=2, max_kv=2, num_heads=2, scale=0.1, causal=1, err_flag=None, workspace=P(), workspace_bytes=1 << 20)
        f.update(kw)
        return B.lib().moe_attn_expanded(ctypes.byref(B.MoeAttnExpandedArgs(**f)), 0, None)

    assert call(T=0, q=None) == call(B=0) == call(max_q=0) == 0
    for kw in (dict(T=-1), dict(S=-1), dict(B=-1), dict(max_q=-1), dict(max_kv=-1), dict(num_heads=0), dict(scale=0.0),
               dict(scale=math.nan), dict(causal=2), dict(q=None), dict(k=None), dict(k_rope=None), dict(v=None),
               dict(o=None), dict(cu_q=None), dict(cu_kv=None), dict(q_ld=-8), dict(rope_ld=-8), dict(o_ld=128),
               dict(o_head_stride=120), dict(o_ld=0)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(B=8193), dict(T=BIG + 1), dict(S=BIG + 1), dict(max_kv=BIG + 1), dict(num_heads=4097),
               dict(T=BIG, max_kv=BIG, o_ld=1 << 20), dict(q_ld=1 << 39), dict(v_head_stride=1 << 39)):
        assert call(**kw) == UNSUPPORTED, kw
    for n in ("q", "k", "k_rope", "v", "o"):
        assert call(**{n: P(8)}) == ALIGNMENT, n
    for n in ("q_ld", "k_ld", "rope_ld", "v_ld", "o_ld", "q_head_stride", "k_head_stride", "v_head_stride"):
        assert call(**{n: 2052}) == ALIGNMENT, n
    assert call(workspace=None) == call(workspace_bytes=100) == WORKSPACE
    assert B.lib().moe_attn_expanded(None, 0, None) == INVALID
    assert B.moe_attn_expanded_workspace_size(16) > 0 and B.moe_attn_expanded_workspace_size(0) == 0


def test_norm_arguments(P):
    def call(**kw):
        f = dict(y=P(), post_weight=P(), gate=P(), resid=P(), resid_out=P(), pre_weight=P(), out=P(), T=2, hidden=64,
                 dtype=B.BF16, resid_dtype=B.F32, gate_rows=1, scale=1.0, eps=1e-6)
        f.update(kw)
        return B.lib().moe_block_norm(ctypes.byref(B.MoeNormArgs(**f)), 0, None)

    assert call(T=0, y=None) == 0
    for kw in (dict(T=-1), dict(hidden=0), dict(y=None), dict(out=None, resid_out=None), dict(pre_weight=None),
               dict(gate_rows=3), dict(gate_rows=0), dict(scale=math.inf), dict(eps=-1.0), dict(eps=math.nan)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(hidden=60), dict(hidden=16392), dict(dtype=B.FP8_E4M3), dict(resid_dtype=B.FP8_E4M3), dict(dtype=9)):
        assert call(**kw) == UNSUPPORTED, kw
    for n in ("y", "post_weight", "gate", "resid", "resid_out", "pre_weight", "out"):
        assert call(**{n: P(8)}) == ALIGNMENT, n
    assert B.lib().moe_block_norm(None, 0, None) == INVALID


def test_the_binding_refuses_other_shapes():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for pool in (torch.zeros(2, 16, 576), bf(2, 16, 512), bf(2, 16, 1152)[:, :, ::2], bf(32, 576)):
        with pytest.raises(ValueError):
            B.latent_cache(pool)
    c = B.latent_cache(bf(2, 16, 576))
    slots = torch.zeros(3, dtype=torch.int64)
    for a, r, s, w in ((bf(3, 500), bf(3, 64), slots, None), (bf(3, 512), bf(2, 64), slots, None),
                       (torch.zeros(3, 512), bf(3, 64), slots, None), (bf(3, 512), bf(3, 64), slots.int(), None),
                       (bf(3, 512), bf(3, 64), slots[:2], None), (bf(3, 512), bf(3, 64), slots, bf(64)),
                       (bf(3, 1024)[:, ::2], bf(3, 64), slots, None), (bf(3, 512), bf(3, 64), slots, torch.zeros(512))):
        with pytest.raises(ValueError):
            B.moe_latent_write(c, a, r, s, weight=w)
    more = (i32(2), i32(1), i32(1, 4), 2, 8, 0.1)
    for q, o in ((bf(2, 4, 512), bf(2, 4, 512)), (bf(2, 4, 576), bf(2, 4, 576)), (bf(2, 4, 576), bf(2, 3, 512)),
                 (torch.zeros(2, 4, 576), bf(2, 4, 512)), (bf(2, 4, 576), torch.zeros(2, 4, 512))):
        with pytest.raises(ValueError):
            B.attn_latent_args(q, o, *more)
    args = B.attn_latent_args(bf(2, 4, 576), bf(2, 4, 512), *more)
    for tree in (i32(2), torch.zeros(3, dtype=torch.int64), torch.zeros(4, dtype=torch.int64)[::2]):
        with pytest.raises(ValueError):
            B.moe_attn_latent(c, args, tree=tree)
    kv = B.kv_cache(bf(2, 2, 16, 64), bf(2, 2, 16, 64))
    with pytest.raises(ValueError):  # heads as wide as the latent cache's
        B.moe_attn_tree(kv, args, torch.zeros(2, dtype=torch.int64))
    paged = B.attn_args(bf(2, 4, 64), bf(2, 4, 64), *more)
    with pytest.raises(ValueError):
        B.moe_attn_latent(c, paged)
    with pytest.raises(ValueError):
        B.moe_attn_tree(kv, paged, torch.zeros(3, dtype=torch.int64))
    good = dict(q=bf(2, 4, 192), k=bf(3, 4, 128), k_rope=bf(3, 64), v=bf(3, 4, 128), o=bf(2, 4, 128), cu_q=i32(2), cu_kv=i32(2))
    B.attn_expanded_args(**good, max_q=2, max_kv=3, scale=0.1)
    for n, t in (("q", bf(2, 4, 128)), ("k", bf(3, 3, 128)), ("k_rope", bf(2, 64)), ("v", bf(3, 4, 64)), ("o", bf(2, 4, 192)),
                 ("cu_kv", i32(3)), ("k", torch.zeros(3, 4, 128)), ("v", bf(3, 4, 256)[:, :, ::2])):
        with pytest.raises(ValueError):
            B.attn_expanded_args(**{**good, n: t}, max_q=2, max_kv=3, scale=0.1)
    with pytest.raises(ValueError):
        B.attn_expanded_args(**good, max_q=2, max_kv=3, scale=0.1, lse=torch.zeros(2, 3))
    y, w = bf(4, 64), bf(64)
    for kw in (dict(y=y.half(), out=y.half(), pre_weight=w.half()), dict(y=bf(4, 128)[:, ::2], out=y, pre_weight=w),
               dict(y=y, out=bf(4, 72), pre_weight=w), dict(y=y, out=y.float(), pre_weight=w),
               dict(y=y, out=y, pre_weight=w.float()), dict(y=y, out=y, pre_weight=bf(72)),
               dict(y=y, out=y, pre_weight=w, resid=y, resid_out=y.float()),
               dict(y=y, out=y, pre_weight=w, gate=bf(3, 64)), dict(y=y, out=y, pre_weight=w, gate=torch.zeros(4, 64)),
               dict(y=y, out=y, pre_weight=w, resid=bf(3, 64))):
        with pytest.raises(ValueError):
            B.moe_block_norm(**kw)


def test_plain_masks_and_trees():
    assert R.chain(2, 4).tolist() == [[True, True, True, False], [True] * 4]
    assert R.chain(3, 2).tolist() == [[False, False], [True, False], [True, True]]
    assert R.chain(2, 4, window=2).tolist() == [[False, True, True, False], [False, False, True, True]]
    for n, kv in ((5, 9), (4, 2), (64, 70)):
        line = np.array([(1 << (i + 1)) - 1 for i in range(n)], dtype=np.uint64)
        assert np.array_equal(R.branches(line, n, kv), R.chain(n, kv))
    t = R.random_tree(np.random.default_rng(0), 64).tolist()
    for i, bits in enumerate(t):
        assert bits >> i == 1  # itself, and none after it
        for j in range(i):
            if bits >> j & 1:
                assert t[j] & ~bits == 0  # an ancestor's ancestors are its own


def test_plain_attention_and_norm_against_torch():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 2, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 4))
    o, lse, _, _ = R.attention(q, k, v, R.chain(3, 5), 0.3)
    s = torch.einsum("nhd,kd->nhk", *map(torch.tensor, (q, k))) * 0.3
    s = s.masked_fill(~torch.tensor(R.chain(3, 5))[:, None], -math.inf)
    assert np.allclose(o, (s.softmax(-1) @ torch.tensor(v)).numpy()) and np.allclose(lse, s.logsumexp(-1).numpy())
    y, w = rng.standard_normal((3, 16)), rng.standard_normal(16)
    r, out = R.block_norm(y, w, resid=y + 1, post=w, gate=y, scale=2.0, eps=0.1)
    t = torch.tensor
    n = lambda x: torch.nn.functional.rms_norm(x, (16,), t(w), 0.1)
    assert np.allclose(r, t(y) + 1 + 2.0 * t(y) * n(t(y))) and np.allclose(out, n(t(r)))


def test_arguments_keep_their_tensors():
    """The structures hold addresses: tensors made for the call alone live as long as they do."""
    import gc
    import weakref

    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    q, cu, ws = bf(2, 4, 576), i32(2), torch.zeros(8)
    refs = [weakref.ref(t) for t in (q, cu, ws)]
    args = B.attn_latent_args(q, bf(2, 4, 512), cu, i32(1), i32(1, 4), 2, 8, 0.1, workspace=ws)
    del q, cu, ws
    gc.collect()
    assert all(r() is not None for r in refs)
    del args
    gc.collect()
    assert all(r() is None for r in refs)
    k = bf(3, 4, 128)
    ref = weakref.ref(k)
    args = B.attn_expanded_args(bf(2, 4, 192), k, bf(3, 64), bf(3, 4, 128), bf(2, 4, 128), i32(2), i32(2), 2, 3, 0.1)
    del k
    gc.collect()
    assert ref() is not None and args.k == ref().data_ptr()
