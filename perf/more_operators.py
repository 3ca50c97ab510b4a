"""Cases of the operators for latent attention, trees of drafted tokens and the norms around a block.

A case is a dict of plain values; ``op`` says which operator it measures:

* ``norm``     -- a block's output normed, gated, scaled and added to the residual, and the next
                  block's input normed from it;
* ``latent``   -- the new tokens' latent vectors (normed) and rotary keys into the pages of a cache;
* ``absorbed`` -- attention of each request's new tokens over such a cache, every head reading the
                  same 576 numbers a token and the first 512 of them as its value; with a tree the
                  new tokens see those of their own branch;
* ``expanded`` -- the same attention for prompts, with keys (128 + 64 shared) and values (128) of
                  every head written out;
* ``tree``     -- attention of a tree of drafted tokens over a cache of grouped heads.

Lengths are a function of the case alone (``lens`` seeds them); values, page tables and trees are a
function of the seed.  ``run`` computes the plain form, or, where ``own`` is true, calls the library.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn
LATENT, ROPE, HEAD = 512, 64, 128  # numbers a token in the latent cache; an expanded head's key and value
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 tokens between attention and experts: the call is all latency
        dict(name="norm_decode_bf16", op="norm", dtype="bf16", resid="bf16", tokens=64, hidden=2048, post=False,
             gate="none"),
        # a large prefill step with a norm on either side of the block, a gate a channel and an fp32 residual
        dict(name="norm_prefill_gated", op="norm", dtype="bf16", resid="f32", tokens=16384, hidden=7168, post=True,
             gate="row"),
        # one decode step of 64 requests: the call is all latency
        dict(name="latent_write_decode", op="latent", tokens=64, norm=True, page=64),
        # the two prompt chunks of a large prefill step
        dict(name="latent_write_prefill", op="latent", tokens=16384, norm=True, page=64),
        # one request decoding on a short context with few heads: the call is all latency
        dict(name="absorbed_one", op="absorbed", requests=1, max_q=1, max_kv=1501, lens=1, heads=16, page=64,
             tree=False),
        # an ordinary decode step of many requests of different ages, 128 heads: memory and tensor cores even
        dict(name="absorbed_decode_wide", op="absorbed", requests=64, max_q=1, max_kv=16384, lens=3, heads=128,
             page=64, tree=False),
        # trees of up to six drafted tokens to be verified, few heads: memory
        dict(name="absorbed_tree_narrow", op="absorbed", requests=48, max_q=6, max_kv=20001, lens=4, heads=16,
             page=32, tree=True),
        # prompts of ragged sizes, some after a prefix
        dict(name="expanded_ragged", op="expanded", requests=7, max_q=1100, max_kv=2311, lens=5, heads=16),
        # one long prompt with many heads: bound by the tensor cores
        dict(name="expanded_long", op="expanded", requests=1, max_q=8192, max_kv=8192, lens=6, heads=128),
        # one request's small tree on a short context: the call is all latency
        dict(name="tree_one_bf16", op="tree", dtype="bf16", requests=1, max_q=13, max_kv=1234, lens=7, q_heads=32,
             kv_heads=4, head_dim=128, page=16),
        # trees of up to eight nodes over small heads of a quantised cache, as the few-row form takes them
        dict(name="tree_small_e4m3", op="tree", dtype="e4m3", requests=40, max_q=8, max_kv=8191, lens=8, q_heads=16,
             kv_heads=8, head_dim=64, page=32),
        # large trees of up to 64 nodes, many rows a key/value head
        dict(name="tree_large_bf16", op="tree", dtype="bf16", requests=32, max_q=64, max_kv=8192, lens=9, q_heads=32,
             kv_heads=4, head_dim=128, page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "latent", "absorbed", "absorbed", "expanded", "tree", "tree"])
    lens = rng.randint(0, 10**6)
    page = rng.choice([16, 32, 64, 128])
    if op == "norm":
        hidden = 8 * _log(rng, 16, 1024)
        return dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), resid=rng.choice(["bf16", "f32"]),
                    tokens=_log(rng, 1, min(32768, (1 << 26) // hidden)), hidden=hidden, post=rng.random() < 0.5,
                    gate=rng.choice(["none", "row", "token"]))
    if op == "latent":
        return dict(op=op, tokens=_log(rng, 1, 16384), norm=rng.random() < 0.7, page=page)
    if op == "expanded":
        n, heads = _log(rng, 1, 16), rng.choice([1, 5, 16, 32, 128])
        max_q = _log(rng, 1, 8192 // n)
        return dict(op=op, requests=n, max_q=max_q, max_kv=_log(rng, max_q, max(max_q, 8192 // n)), lens=lens,
                    heads=heads)
    if op == "absorbed":
        heads = rng.choice([8, 16, 20, 64, 96, 128])
        n = _log(rng, 1, 128)
        max_q = rng.choice([1, 1, rng.randint(2, 8), rng.randint(9, 64)])
        max_q = min(max_q, max(1, 1024 // n))
        cap = min(32768, (1 << 20) // n, (1 << 27) // (n * max_q * heads))
        return dict(op=op, requests=n, max_q=max_q, max_kv=_log(rng, max_q, max(cap, max_q + 1)), lens=lens,
                    heads=heads, page=page, tree=max_q > 1 and rng.random() < 0.5)
    kv_heads = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    n, max_q = _log(rng, 1, 64), rng.randint(1, 64)
    cap = min(32768, (1 << 28) // (n * max_q * kv_heads * group), (1 << 19) // n)
    return dict(op=op, dtype=rng.choice(["bf16", "e4m3"]), requests=n, max_q=max_q,
                max_kv=_log(rng, max_q, max(cap, max_q + 1)), lens=lens, q_heads=kv_heads * group, kv_heads=kv_heads,
                head_dim=rng.choice([64, 128]), page=page)


def _lens(case):
    """(q_len, kv_len) of an attention case's requests: the first one has the largest of both."""
    rng = random.Random(case["lens"])
    q, kv = [case["max_q"]], [case["max_kv"]]
    for _ in range(case["requests"] - 1):
        n = rng.randint(1, case["max_q"])
        q.append(n)
        kv.append(rng.randint(n, case["max_kv"]))
    return q, kv


# ----------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return g


def _randn(g, *shape, dtype=torch.bfloat16, std=1.0):
    return torch.empty(shape, dtype=dtype, device=DEV).normal_(std=std, generator=g)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _i32([0] + np.cumsum(lens).tolist())


def _table(lens, page, g):
    """Pages of each request, scattered over the pool: (pages in the pool, [requests][width] int32)."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 3
    perm = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor(np.cumsum([0] + need[:-1]), device=DEV)
    width = max(max(need), 1)
    at = first[:, None] + torch.arange(width, device=DEV)[None]
    inside = torch.arange(width, device=DEV)[None] < torch.tensor(need, device=DEV)[:, None]
    return pages, torch.where(inside, perm[at.clamp(max=pages - 1)], 0).contiguous()


def _trees(q_len, seed):
    """A tree of each request's new tokens: int64 [T], bit j of a token says that it sees its request's
    j-th new token, which is itself or one that it descends from."""
    rng = np.random.default_rng(seed)
    out = []
    for n in q_len:
        mine = []
        for i in range(n):
            # a drafted tree is bushy near its root: the parent is one of the last few nodes or none
            parent = int(rng.integers(max(-1, i - 6), i)) if i else -1
            mine.append((mine[parent] if parent >= 0 else 0) | 1 << i)
        out += mine
    return torch.from_numpy(np.array(out, dtype=np.uint64).view(np.int64)).to(DEV)


def _library():
    from moe_expert_dispatch_route_gb300 import binding

    return binding


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "norm":
        T, H = case["tokens"], case["hidden"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        rt = torch.float32 if case["resid"] == "f32" else torch.bfloat16
        st.update(y=_randn(g, T, H, dtype=dt, std=0.7), resid=_randn(g, T, H, dtype=rt, std=2.0))
        st["pre"] = 1 + _randn(g, H, dtype=dt, std=0.2)
        st["post"] = 1 + _randn(g, H, dtype=dt, std=0.2) if case["post"] else None
        st["gate"] = None if case["gate"] == "none" else _randn(g, 1 if case["gate"] == "row" else T, H, dtype=dt)
        st.update(scale=0.75, resid_out=torch.empty_like(st["resid"]), out=torch.empty_like(st["y"]))
    elif op == "latent":
        T, page = case["tokens"], case["page"]
        pages = -(-T // page) + 3
        # the projection's output: the latent vector and the rotary key of a token side by side
        down = _randn(g, T, LATENT + ROPE)
        st.update(c=down[:, :LATENT], k_rope=down[:, LATENT:])
        st["weight"] = 1 + _randn(g, LATENT, std=0.2) if case["norm"] else None
        st["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:T].contiguous()
        st["pool"] = _randn(g, pages, page, LATENT + ROPE)
    else:
        q_len, kv_len = _lens(case)
        T = sum(q_len)
        st["cu"] = _cu(q_len)
        if op == "expanded":
            S, H = sum(kv_len), case["heads"]
            st.update(q=_randn(g, T, H, HEAD + ROPE), k_rope=_randn(g, S, ROPE), cu_kv=_cu(kv_len))
            # the up projection's output holds keys and values of a head side by side
            up = _randn(g, S, H, 2 * HEAD)
            st.update(k=up[..., :HEAD], v=up[..., HEAD:], scale=(HEAD + ROPE)**-0.5)
            st.update(o=torch.empty(T, H, HEAD, dtype=torch.bfloat16, device=DEV))
        else:
            pages, st["table"] = _table(kv_len, case["page"], g)
            st["kv_len"] = _i32(kv_len)
            st["tree"] = _trees(q_len, seed * 31 + 7) if op == "tree" or case["tree"] else None
            if op == "absorbed":
                H = case["heads"]
                st["pool"] = _randn(g, pages, case["page"], LATENT + ROPE)
                # queries after the key's up projection: scores of a few units, as the model's own scale leaves them
                st.update(q=_randn(g, T, H, LATENT + ROPE, std=0.7), scale=(HEAD + ROPE)**-0.5)
                st.update(o=torch.empty(T, H, LATENT, dtype=torch.bfloat16, device=DEV))
            else:
                H, D = case["q_heads"], case["head_dim"]
                shape = (pages, case["kv_heads"], case["page"], D)
                for n in ("k", "v"):
                    if case["dtype"] == "bf16":
                        st[n], st[n + "_scale"] = _randn(g, *shape), None
                    else:
                        st[n] = _randn(g, *shape, std=120.0).clamp_(-448, 448).to(E4M3)
                        st[n + "_scale"] = torch.randint(118, 123, shape[:3], generator=g, device=DEV, dtype=torch.uint8)
                st.update(q=_randn(g, T, H, D), scale=D**-0.5)
                st.update(o=torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV))
        st["lse"] = torch.empty(T, H, dtype=torch.float32, device=DEV)
    if own:
        st["lib"] = lib = _library()
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        size = 0
        if op in ("latent", "absorbed"):
            st["cache"] = lib.latent_cache(st["pool"])
        if op == "absorbed":
            size = lib.moe_attn_latent_workspace_size(st["cache"], case["heads"])
        elif op == "expanded":
            size = lib.moe_attn_expanded_workspace_size(case["heads"])
        elif op == "tree":
            st["cache"] = lib.kv_cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
            size = lib.moe_attn_workspace_size(st["cache"], case["q_heads"])
        if size:
            st["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
            more = dict(lse=st["lse"], workspace=st["ws"], err_flag=st["err"])
            if op == "expanded":
                st["args"] = lib.attn_expanded_args(st["q"], st["k"], st["k_rope"], st["v"], st["o"], st["cu"],
                                                    st["cu_kv"], case["max_q"], case["max_kv"], st["scale"], **more)
            else:
                build = lib.attn_latent_args if op == "absorbed" else lib.attn_args
                st["args"] = build(st["q"], st["o"], st["cu"], st["kv_len"], st["table"], case["max_q"],
                                   case["max_kv"], st["scale"], **more)
    return st


# ------------------------------------------------------------------------------ one pass
def run(state):
    return {"norm": _norm, "latent": _latent, "absorbed": _absorbed, "expanded": _expanded,
            "tree": _tree}[state["case"]["op"]](state)


def _rms(x, w):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.float()


def _norm(st):
    if own:
        st["lib"].moe_block_norm(st["y"], st["out"], st["pre"], resid=st["resid"], resid_out=st["resid_out"],
                                 post_weight=st["post"], gate=st["gate"], scale=st["scale"], eps=EPS)
        return [st["resid_out"], st["out"]]
    x = st["y"].float()
    if st["post"] is not None:
        x = _rms(x, st["post"])
    if st["gate"] is not None:
        x = x * st["gate"].float()
    r = st["resid"].float() + st["scale"] * x
    return [r.to(st["resid"].dtype), _rms(r, st["pre"]).to(st["y"].dtype)]


def _latent(st):
    if own:
        st["lib"].moe_latent_write(st["cache"], st["c"], st["k_rope"], st["slots"], weight=st["weight"], eps=EPS,
                                   err_flag=st["err"])
        return st["pool"]
    c = st["c"].float()
    if st["weight"] is not None:
        c = _rms(c, st["weight"])
    page, at = st["slots"] // st["case"]["page"], st["slots"] % st["case"]["page"]
    st["pool"][page, at] = torch.cat([c.to(torch.bfloat16), st["k_rope"]], 1)
    return st["pool"]


def _padded(st, Q, T):
    """Rows of q padded to the longest request, and back: (at [B][Q], (b, t) of the packed rows)."""
    at = (st["cu"][:-1, None] + torch.arange(Q, device=DEV)[None]).clamp(max=T - 1)
    row = torch.arange(T, device=DEV, dtype=torch.int32)
    b = torch.searchsorted(st["cu"][1:], row, right=True)
    return at, b, (row - st["cu"][b]).long()


def _seen(st, at, n, kv_len, K):
    """Which keys each padded row sees [B][Q][K]: cached ones before it, or those of its branch."""
    i, j = torch.arange(at.shape[1], device=DEV), torch.arange(K, device=DEV)
    first = (kv_len - n)[:, None, None]
    new = j[None, None] - first
    if st.get("tree") is None:
        return (new <= i[None, :, None]) & (j[None, None] < kv_len[:, None, None])
    bits = st["tree"][at][..., None] >> new.clamp(0, 63)
    return (new < 0) | (((bits & 1) == 1) & (new < n[:, None, None]))


def _softmax(s, seen):
    """Probabilities before their division, their sum and the logarithm of the whole sum."""
    s.masked_fill_(~seen, -math.inf)
    m = s.amax(-1, keepdim=True)
    s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = s.sum(-1, keepdim=True)
    return s, total, m[..., 0] + total[..., 0].log()


def _absorbed(st):
    if own:
        st["lib"].moe_attn_latent(st["cache"], st["args"], tree=st["tree"])
        return [st["o"], st["lse"]]
    c = st["case"]
    B, Q, K, H = c["requests"], c["max_q"], c["max_kv"], c["heads"]
    T = st["q"].shape[0]
    at, b, t = _padded(st, Q, T)
    j = torch.arange(K, device=DEV)
    keys = st["pool"][st["table"].long()[:, j // c["page"]], (j % c["page"])[None].expand(B, K)].float()
    q = st["q"].float()[at].reshape(B, Q * H, LATENT + ROPE)
    s = (q @ keys.transpose(1, 2)).view(B, Q, H, K) * st["scale"]
    seen = _seen(st, at, st["cu"][1:] - st["cu"][:-1], st["kv_len"], K)
    s, total, lse = _softmax(s, seen[:, :, None])
    v = torch.where((j[None] < st["kv_len"][:, None])[..., None], keys[..., :LATENT], 0.0)
    o = (s.view(B, Q * H, K) @ v).view(B, Q, H, LATENT) / total
    return [o[b, t].to(torch.bfloat16), lse[b, t]]


def _expanded(st):
    if own:
        st["lib"].moe_attn_expanded(st["args"])
        return [st["o"], st["lse"]]
    c = st["case"]
    B, Q, K, H = c["requests"], c["max_q"], c["max_kv"], c["heads"]
    T, S = st["q"].shape[0], st["k_rope"].shape[0]
    at, b, t = _padded(st, Q, T)
    n, kv_len = st["cu"][1:] - st["cu"][:-1], st["cu_kv"][1:] - st["cu_kv"][:-1]
    key = (st["cu_kv"][:-1, None] + torch.arange(K, device=DEV)[None]).clamp(max=S - 1)
    q = st["q"].float()[at].transpose(1, 2)
    k = torch.cat([st["k"].float(), st["k_rope"].float()[:, None].expand(S, H, ROPE)], 2)[key].permute(0, 2, 3, 1)
    s, total, lse = _softmax((q @ k).mul_(st["scale"]), _seen(st, at, n, kv_len, K)[:, None])
    del k
    o = (s @ st["v"].float()[key].transpose(1, 2)).div_(total)
    return [o.transpose(1, 2)[b, t].to(torch.bfloat16), lse.transpose(1, 2)[b, t]]


def _scaled(st, n, page, at):
    """Cached tokens as numbers: [..., heads, head_dim] in 32 bits."""
    if st["k_scale"] is None:
        return st[n][page, :, at].float()
    codes = st[n].view(torch.uint8)[page, :, at].view(E4M3).float()
    return torch.ldexp(codes, st[n + "_scale"][page, :, at].int()[..., None] - 127)


def _tree(st):
    if own:
        st["lib"].moe_attn_tree(st["cache"], st["args"], st["tree"])
        return [st["o"], st["lse"]]
    c = st["case"]
    B, Q, K, H, G, D = c["requests"], c["max_q"], c["max_kv"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    T = st["q"].shape[0]
    at, b, t = _padded(st, Q, T)
    j = torch.arange(K, device=DEV)
    page, slot = st["table"].long()[:, j // c["page"]], (j % c["page"])[None].expand(B, K)
    q = st["q"].float()[at].view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    s = (q @ _scaled(st, "k", page, slot).permute(0, 2, 3, 1)).view(B, H, G, Q, K) * st["scale"]
    seen = _seen(st, at, st["cu"][1:] - st["cu"][:-1], st["kv_len"], K)
    s, total, lse = _softmax(s, seen[:, None, None])
    v = torch.where((j[None] < st["kv_len"][:, None])[..., None, None], _scaled(st, "v", page, slot), 0.0)
    o = (s.view(B, H, G * Q, K) @ v.permute(0, 2, 1, 3)).view(B, H, G, Q, D) / total
    return [o.permute(0, 3, 1, 2, 4)[b, t].reshape(T, H * G, D).to(torch.bfloat16),
            lse.permute(0, 3, 1, 2)[b, t].reshape(T, H * G)]


# ------------------------------------------------------------------------------- the work
def work(case):
    op = case["op"]
    if op == "norm":
        T, H = case["tokens"], case["hidden"]
        el, rl = (4 if case[n] == "f32" else 2 for n in ("dtype", "resid"))
        rows = {"none": 0, "row": 1, "token": T}[case["gate"]] + 1 + case["post"]
        return {"bytes": T * H * 2 * (el + rl) + rows * H * el, "flops": T * H * (7 + 3 * case["post"])}
    if op == "latent":
        row = 2 * (LATENT + ROPE)
        return {"bytes": case["tokens"] * (2 * row + 8), "flops": 4 * case["tokens"] * LATENT * case["norm"]}
    q, kv = _lens(case)
    T = sum(q)
    # a tree's nodes see as many cached tokens as a chain's, and at least themselves of the new ones
    chain = op == "expanded" or (op == "absorbed" and not case["tree"])
    pairs = sum(m * (n - m) + (m * (m + 1) // 2 if chain else m) for m, n in zip(q, kv))
    if op == "absorbed":
        H = case["heads"]
        return {"bytes": sum(kv) * 2 * (LATENT + ROPE) + T * H * (2 * (2 * LATENT + ROPE) + 4),
                "flops": 2 * H * pairs * (2 * LATENT + ROPE)}
    if op == "expanded":
        H = case["heads"]
        return {"bytes": sum(kv) * 2 * (2 * HEAD * H + ROPE) + T * H * (2 * (2 * HEAD + ROPE) + 4),
                "flops": 2 * H * pairs * (2 * HEAD + ROPE)}
    H, D = case["kv_heads"], case["head_dim"]
    row = 2 * H * (2 * D if case["dtype"] == "bf16" else D + 1)
    return {"bytes": sum(kv) * row + T * (case["q_heads"] * (4 * D + 4) + 8), "flops": 4 * D * case["q_heads"] * pairs}


# ------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]

    def normed(x, w):
        return x / torch.sqrt(x.square().sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.double()

    if op == "norm":
        r, out = [], []
        for rows in torch.arange(case["tokens"], device=DEV).split(2048):
            x = st["y"][rows].double()
            x = x if st["post"] is None else normed(x, st["post"])
            if st["gate"] is not None:
                x = x * (st["gate"] if st["gate"].shape[0] == 1 else st["gate"][rows]).double()
            x = x * st["scale"] + st["resid"][rows].double()
            r.append(x)
            out.append(normed(x, st["pre"]))
        return [torch.cat(r), torch.cat(out)]
    if op == "latent":
        pool = st["pool"].double().flatten(0, 1)
        c = st["c"].double()
        pool[st["slots"], :LATENT] = c if st["weight"] is None else normed(c, st["weight"])
        pool[st["slots"], LATENT:] = st["k_rope"].double()
        return pool.view(st["pool"].shape)
    q_len, kv_len = _lens(case)
    heads = case["q_heads"] if op == "tree" else case["heads"]
    o, lse, a, e = [], [], 0, 0
    for b, (m, n) in enumerate(zip(q_len, kv_len)):
        hidden = torch.ones(m, n, dtype=torch.bool, device=DEV).triu(n - m + 1)
        if st.get("tree") is not None:
            hidden = torch.zeros_like(hidden)
            for i, bits in enumerate(st["tree"][a:a + m].tolist()):
                for j in range(m):
                    hidden[i, n - m + j] = not bits >> j & 1
        if op != "expanded":
            pages = st["table"][b, :-(-n // case["page"])].long()
        if op == "absorbed":
            keys = st["pool"][pages].flatten(0, 1)[:n].double()
        elif op == "tree":
            kv = []
            for name in ("k", "v"):
                x = st[name][pages].double()
                if st["k_scale"] is not None:
                    x = x * torch.exp2(st[name + "_scale"][pages].double() - 127)[..., None]
                kv.append(x.transpose(1, 2).flatten(0, 1)[:n])
        for_h, lse_h = [], []
        for h in range(heads):
            x = st["q"][a:a + m, h].double()
            if op == "absorbed":
                k, v = keys, keys[:, :LATENT]
            elif op == "expanded":
                k = torch.cat([st["k"][e:e + n, h], st["k_rope"][e:e + n]], 1).double()
                v = st["v"][e:e + n, h].double()
            else:
                k, v = (x_[:, h // (heads // case["kv_heads"])] for x_ in kv)
            w = torch.einsum("md,nd->mn", x, k) * st["scale"]
            w.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(w, -1)
            for_h.append(w.sub_(z[:, None]).exp_() @ v)
            lse_h.append(z)
        o.append(torch.stack(for_h, 1))
        lse.append(torch.stack(lse_h, 1))
        a, e = a + m, e + n
    return [torch.cat(o), torch.cat(lse)]
