"""Strides of an index that has one value are not used: tensors that have odd ones are served like packed ones."""
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B

WORKSPACE = 4
BF16 = torch.bfloat16


def odd(rows, heads, width, device="cpu"):
    """[rows][heads][width] whose strides of single rows or heads are odd, its rows aligned."""
    ld = 1001 if rows == 1 else heads * 1000
    hs = 997 if heads == 1 else 1000
    base = torch.zeros(16 + rows * ld + heads * hs + width, dtype=BF16, device=device)
    first = -(base.data_ptr() // 2) % 8  # elements to the next 16-byte boundary
    return base.as_strided((rows, heads, width), (ld, hs, 1), first)


@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 4), (3, 1), (1, 16)])
def test_the_binding_takes_any_unused_stride(rows, heads):
    """(A call that gets as far as its workspace has passed every other check.)"""
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    bf = lambda *s: torch.zeros(*s, dtype=BF16)
    more = (i32(2), i32(1), i32(1, 4), rows, 8, 0.1)

    def refused_for_its_workspace(call):
        with pytest.raises(B.MoeError) as e:
            call()
        assert e.value.status == WORKSPACE

    latent = B.latent_cache(bf(4, 16, 576))
    args = B.attn_latent_args(odd(rows, heads, 576), odd(rows, heads, 512), *more)
    refused_for_its_workspace(lambda: B.moe_attn_latent(latent, args, stream=0))
    cache = B.kv_cache(bf(4, 1, 16, 64), bf(4, 1, 16, 64))
    args2 = B.attn_args(odd(rows, heads, 64), odd(rows, heads, 64), *more)
    refused_for_its_workspace(lambda: B.moe_attn_paged(cache, args2, stream=0))
    for keys in (1, 5):
        rope = torch.zeros(8 * 64 + 64, dtype=BF16)
        rope = rope.as_strided((keys, 64), (65 if keys == 1 else 64, 1), -(rope.data_ptr() // 2) % 8)
        args3 = B.attn_expanded_args(odd(rows, heads, 192), odd(keys, heads, 128), rope, odd(keys, heads, 128),
                                     odd(rows, heads, 128), i32(2), i32(2), rows, keys, 0.1)
        refused_for_its_workspace(lambda: B.moe_attn_expanded(args3, stream=0))
    # a stride that is used is still to be a multiple of 16 bytes
    q = torch.zeros(4000, dtype=BF16).as_strided((2, heads, 576), (heads * 576 + 1, 576, 1)) if heads == 1 else None
    if q is not None:
        with pytest.raises(B.MoeError) as e:
            B.moe_attn_latent(latent, B.attn_latent_args(q, bf(2, heads, 512), i32(2), i32(1), i32(1, 4), 2, 8, 0.1),
                              stream=0)
        assert e.value.status == 3


@pytest.mark.gpu
@pytest.mark.parametrize("rows,heads", [(1, 1), (1, 128), (4, 1), (1, 20)])
def test_results_are_those_of_packed_tensors(rows, heads):
    g = torch.Generator(device="cuda").manual_seed(rows * heads)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    packed = lambda *s: torch.empty(*s, dtype=BF16, device="cuda")
    copy = lambda t: odd(*t.shape, device="cuda").copy_(t)
    kv, err = 150, i32([0])
    pool = rand(3, 64, 576)
    cache = B.latent_cache(pool)
    q = rand(rows, heads, 576)
    ws = torch.zeros(B.moe_attn_latent_workspace_size(cache, heads), dtype=torch.uint8, device="cuda")
    got = []
    for a, o in ((q, packed(rows, heads, 512)), (copy(q), odd(rows, heads, 512, "cuda"))):
        B.moe_attn_latent(cache, B.attn_latent_args(a, o, i32([0, rows]), i32([kv]), i32([[2, 0, 1]]), rows, kv, 0.1,
                                                    workspace=ws, err_flag=err))
        got.append(o)
    assert torch.equal(*got)
    for keys in (1, 70):
        q, k, v, r = rand(rows, heads, 192), rand(keys, heads, 128), rand(keys, heads, 128), rand(keys, 64)
        got = []
        for f, o in ((lambda t: t, packed(rows, heads, 128)), (copy, odd(rows, heads, 128, "cuda"))):
            B.moe_attn_expanded(B.attn_expanded_args(f(q), f(k), r, f(v), o, i32([0, rows]), i32([0, keys]), rows, keys, 0.1,
                                                     workspace=ws, err_flag=err))
            got.append(o)
        assert torch.equal(*got)
    pools = rand(2, 3, 1, 64, 64)
    kvc = B.kv_cache(pools[0], pools[1])
    q = rand(rows, min(heads, 32), 64)
    ws = torch.zeros(B.moe_attn_workspace_size(kvc, q.shape[1]), dtype=torch.uint8, device="cuda")
    got = []
    for a, o in ((q, torch.empty_like(q)), (copy(q), odd(*q.shape, "cuda"))):
        B.moe_attn_paged(kvc, B.attn_args(a, o, i32([0, rows]), i32([kv]), i32([[2, 0, 1]]), rows, kv, 0.1, workspace=ws,
                                          err_flag=err))
        got.append(o)
    assert torch.equal(*got) and int(err.item()) == 0
