"""Attention of sharp softmaxes and of maxima that move with every tile, on inputs whose scores are exact (exact_ref.py):
the running maximum's rescaling in every kernel, on one CTA and on pairs, whole and split over CTAs."""
import numpy as np
import pytest
import torch

import exact_ref as X
from latent_ref import branches, chain, random_tree
from moe_expert_dispatch_route_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16 = torch.bfloat16
KINDS = list(X.LATENT)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def paged(values, page, rng):
    """A pool [pages][page][...] of the requests' values in scattered pages, NaN elsewhere, and the table."""
    need = [-(-len(x) // page) for x in values]
    perm = rng.permutation(sum(need) + 2)
    pool = np.full((len(perm) * page, *values[0].shape[1:]), np.nan)
    table = np.zeros((len(values), max(need)), dtype=np.int32)
    at = 0
    for b, x in enumerate(values):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        j = np.arange(len(x))
        pool[table[b, j // page].astype(np.int64) * page + j % page] = x
    return torch.tensor(pool.reshape(len(perm), page, *values[0].shape[1:])), torch.tensor(table, device=DEV)


def masks(rng, tree, n, kv):
    if not tree:
        return chain(n, kv), None
    bits = random_tree(rng, n)
    return branches(bits, n, kv), bits


def tree_of(bits):
    return None if bits[0] is None else torch.from_numpy(np.concatenate(bits).view(np.int64)).to(DEV)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_lens,heads", [([1, 3, 1], 5), ([4, 1, 2], 16), ([1, 2, 1], 20), ([1, 1, 1], 128), ([2, 1, 1], 97),
                                          ([9, 1, 30], 16), ([3, 1, 2], 40)])
@pytest.mark.parametrize("tree,max_ctas", [(False, 0), (True, 0), (False, 2)])
def test_absorbed(kind, q_lens, heads, tree, max_ctas):
    """(Up to 64 rows a request: one CTA; more: pairs, by tokens up to 64 heads, by heads above.)"""
    rng = np.random.default_rng(heads)
    kv_lens = [1290, 70, 400]
    parts = [X.latent_numbers(rng, kind, n, heads, kv) for n, kv in zip(q_lens, kv_lens)]
    seen, bits = zip(*(masks(rng, tree, n, kv) for n, kv in zip(q_lens, kv_lens)))
    pool, table = paged([k for _, k, _, _ in parts], 64, rng)
    pool = pool.to(BF16).to(DEV)
    cache = B.latent_cache(pool)
    q = torch.tensor(np.concatenate([x[0] for x in parts])).to(BF16).to(DEV)
    o = torch.empty(len(q), heads, 512, dtype=BF16, device=DEV)
    lse, err = torch.empty(len(q), heads, device=DEV), i32([0])
    ws = torch.zeros(B.moe_attn_latent_workspace_size(cache, heads), dtype=torch.uint8, device=DEV)
    args = B.attn_latent_args(q, o, i32([0] + np.cumsum(q_lens).tolist()), i32(kv_lens), table, max(q_lens), max(kv_lens),
                              parts[0][3], lse=lse, workspace=ws, err_flag=err)
    B.moe_attn_latent(cache, args, tree=tree_of(bits), max_ctas=max_ctas)
    check(o, lse, err, [X.attention(x[0], x[1], x[2], s, x[3]) for x, s in zip(parts, seen)], q_lens)


def check(o, lse, err, refs, q_lens):
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    o, lse, at = o.double().cpu().numpy(), lse.double().cpu().numpy(), 0
    for b, (ref, n) in enumerate(zip(refs, q_lens)):
        X.check(o[at:at + n], lse[at:at + n], ref, f"request {b}")
        at += n


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_lens,kv_lens", [([70, 200], [1290, 200]), ([300, 1, 129], [300, 1400, 700])])
@pytest.mark.parametrize("causal,max_ctas", [(True, 0), (False, 0), (True, 1)])
def test_expanded(kind, q_lens, kv_lens, causal, max_ctas):
    rng, heads = np.random.default_rng(1), 2
    parts = [[X.latent_numbers(rng, kind, n, 1, kv, 192, 128) for _ in range(heads)] for n, kv in zip(q_lens, kv_lens)]
    ropes = [x[0][1][:, 128:] for x in parts]  # of all heads: the first one's
    cat = lambda f: torch.tensor(np.concatenate([np.stack([f(x) for x in p], 1) for p in parts])).to(BF16).to(DEV)
    q, k, v = cat(lambda x: x[0][:, 0]), cat(lambda x: x[1][:, :128]), cat(lambda x: x[2])
    rope = torch.tensor(np.concatenate(ropes)).to(BF16).to(DEV)
    o, lse, err = torch.empty(len(q), heads, 128, dtype=BF16, device=DEV), torch.empty(len(q), heads, device=DEV), i32([0])
    ws = torch.zeros(B.moe_attn_expanded_workspace_size(heads), dtype=torch.uint8, device=DEV)
    cu = lambda v: i32([0] + np.cumsum(v).tolist())
    scale = parts[0][0][3]
    B.moe_attn_expanded(B.attn_expanded_args(q, k, rope, v, o, cu(q_lens), cu(kv_lens), max(q_lens), max(kv_lens), scale,
                                             causal=causal, lse=lse, workspace=ws, err_flag=err), max_ctas=max_ctas)
    for h in range(heads):
        refs = [X.attention(p[h][0], np.concatenate([p[h][1][:, :128], r], 1), p[h][2], chain(n, kv, causal), scale)
                for p, r, n, kv in zip(parts, ropes, q_lens, kv_lens)]
        check(o[:, h:h + 1], lse[:, h:h + 1], err, refs, q_lens)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("q_lens,heads", [([2, 1, 4], (8, 2)), ([3, 8, 1], (8, 2)), ([8, 1, 5], (16, 4)), ([60, 1, 13], (8, 2))])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_trees(kind, q_lens, heads, D, dtype):
    """(Few rows a key/value head, and tiles.)  Numbers that e4m3 holds, under scales of their own there."""
    rng, kv_lens, (Hq, H) = np.random.default_rng(D), [1290, 70, 400], heads
    a, b, scale, steps, order = X.LATENT[kind]
    steps = min(steps, 4)  # whole numbers up to 15: four bits
    scale *= 4
    if order == "both":
        steps = 3
    vals = [[[X.growing(X.whole(rng, kv, D, most=b), steps, order) for _ in range(H)] for kv in kv_lens] for _ in range(2)]
    q = [X.whole(rng, n, Hq, D, most=a) for n in q_lens]
    seen, bits = zip(*(masks(rng, True, n, kv) for n, kv in zip(q_lens, kv_lens)))
    pools, scales = [], []
    state = np.random.default_rng(7).bit_generator.state
    for x in vals:  # the same pages for keys and values
        r = np.random.default_rng()
        r.bit_generator.state = state
        pool, table = paged([np.stack(y, 1) for y in x], 32, r)  # [pages][page][H][D]
        pool = pool.permute(0, 2, 1, 3).contiguous()
        if dtype == "e4m3":
            byte = torch.randint(125, 130, pool.shape[:3], generator=torch.Generator().manual_seed(3))
            pool = torch.ldexp(pool, 127 - byte[..., None]).to(torch.float8_e4m3fn)
            scales.append(byte.to(torch.uint8).to(DEV))
        pools.append((pool if dtype == "e4m3" else pool.to(BF16)).to(DEV))
    cache = B.kv_cache(*pools, *scales)
    qd = torch.tensor(np.concatenate(q)).to(BF16).to(DEV)
    o, lse, err = torch.empty_like(qd), torch.empty(len(qd), Hq, device=DEV), i32([0])
    ws = torch.zeros(B.moe_attn_workspace_size(cache, Hq), dtype=torch.uint8, device=DEV)
    B.moe_attn_tree(cache, B.attn_args(qd, o, i32([0] + np.cumsum(q_lens).tolist()), i32(kv_lens), table, max(q_lens),
                                       max(kv_lens), scale, lse=lse, workspace=ws, err_flag=err), tree_of(bits))
    G = Hq // H
    for h in range(H):
        refs = [X.attention(q[i][:, h * G:(h + 1) * G], vals[0][i][h], vals[1][i][h], seen[i], scale)
                for i in range(len(q_lens))]
        if dtype == "e4m3":
            # the weights of these caches are fp16: p 2^(b - ref) 2^7 to a multiple of 2^-24, so o is off by 2^-25 2^-7 of
            # every seen value at the reference scale, here the largest: 2^4 times the value at most.  2^-28 |v| a key, in
            # units of what check() multiplies by 2^-8
            refs = [(o_, l_, mag + 2.0**-20 * (s_.astype(float) @ np.abs(vals[1][i][h]))[:, None], e_)
                    for i, ((o_, l_, mag, e_), s_) in enumerate(zip(refs, seen))]
        check(o[:, h * G:(h + 1) * G], lse[:, h * G:(h + 1) * G], err, refs, q_lens)
