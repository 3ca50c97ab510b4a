"""Cases of the serving operators around the MoE layer: the paged key/value cache (written, read
back, attended over) and the verification of drafted tokens.

A case is a dict of plain values; ``op`` says which operator it measures:

* ``write``  -- the new tokens' keys and values into the pages of a cache (bf16, or e4m3 with one
  power-of-two scale per token and head);
* ``read``   -- ranges of cached tokens back to packed bf16 rows;
* ``attend`` -- attention of each request's new tokens (one, a draft, a prompt chunk) over its
  pages, with grouped heads, causal, optionally in a sliding window;
* ``verify`` -- acceptance of drafted tokens against the target's probabilities from given
  uniform numbers, and the token drawn in place of the first one that is refused.

Lengths are a function of the case alone (``lens`` seeds them); values, page tables and random
numbers are a function of the seed.  ``run`` computes the plain form, or, where ``own`` is true,
calls the library.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3 = torch.float8_e4m3fn


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of 64 requests: the call is all latency
        dict(name="write_decode_bf16", op="write", dtype="bf16", tokens=64, kv_heads=4, head_dim=128, page=16),
        # the two prompt chunks of a large prefill step, quantised as they are written
        dict(name="write_prefill_e4m3", op="write", dtype="e4m3", tokens=16384, kv_heads=8, head_dim=128, page=64),
        # a few odd prefixes of small heads, read back for a dense consumer
        dict(name="read_ragged_bf16", op="read", dtype="bf16", requests=13, max_len=700, lens=5, kv_heads=2,
             head_dim=64, page=32),
        # long quantised prefixes taken out of the cache, to be sent or kept elsewhere
        dict(name="read_long_e4m3", op="read", dtype="e4m3", requests=4, max_len=32768, lens=2, kv_heads=8,
             head_dim=128, page=64),
        # one request decoding on a short context: the call is all latency
        dict(name="decode_one_bf16", op="attend", dtype="bf16", requests=1, max_q=1, max_kv=777, lens=1, q_heads=32,
             kv_heads=4, head_dim=128, page=16, window=0),
        # an ordinary decode step: many requests of very different ages, read once at memory speed
        dict(name="decode_ragged_bf16", op="attend", dtype="bf16", requests=128, max_q=1, max_kv=16384, lens=3,
             q_heads=32, kv_heads=4, head_dim=128, page=64, window=0),
        # the same on a quantised cache
        dict(name="decode_ragged_e4m3", op="attend", dtype="e4m3", requests=96, max_q=1, max_kv=20001, lens=4,
             q_heads=64, kv_heads=8, head_dim=128, page=32, window=0),
        # drafts of up to six tokens to be verified, small heads, sliding window
        dict(name="draft_window_bf16", op="attend", dtype="bf16", requests=32, max_q=6, max_kv=8191, lens=6,
             q_heads=40, kv_heads=8, head_dim=64, page=16, window=4096),
        # prompt chunks of ragged sizes beside short ones, on a quantised cache
        dict(name="chunks_ragged_e4m3", op="attend", dtype="e4m3", requests=8, max_q=512, max_kv=8200, lens=7,
             q_heads=32, kv_heads=4, head_dim=128, page=64, window=0),
        # one large prompt chunk on top of as long a prefix: bound by the tensor cores
        dict(name="prefill_long_bf16", op="attend", dtype="bf16", requests=1, max_q=8192, max_kv=16384, lens=8,
             q_heads=32, kv_heads=4, head_dim=128, page=64, window=0),
        # one request's draft: the call is all latency
        dict(name="verify_one", op="verify", dtype="f32", requests=1, max_draft=4, lens=9, vocab=32001),
        # a large batch with a large vocabulary
        dict(name="verify_batch", op="verify", dtype="f32", requests=256, max_draft=4, lens=10, vocab=131072),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "verify"])
    if op == "verify":
        return dict(op=op, dtype=rng.choice(["f32", "bf16"]), requests=_log(rng, 1, 256), max_draft=rng.randint(1, 6),
                    lens=rng.randint(0, 10**6), vocab=_log(rng, 1000, 131072))
    head_dim = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["bf16", "e4m3"])
    kv_heads = rng.choice([1, 2, 4, 8])
    if op == "write":
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 16384), kv_heads=kv_heads, head_dim=head_dim, page=page)
    if op == "read":
        n = _log(rng, 1, 32)
        return dict(op=op, dtype=dtype, requests=n, max_len=_log(rng, 1, 131072 // n), lens=rng.randint(0, 10**6),
                    kv_heads=kv_heads, head_dim=head_dim, page=page)
    kind = rng.choice(["decode", "draft", "chunk"])
    group = rng.choice([1, 2, 4, 5, 7, 8, 16])
    group = max(1, min(group, 64 // kv_heads))
    if kind == "chunk":
        n = _log(rng, 1, 8)
        max_q = _log(rng, 16, 4096 // n)
    else:
        n = _log(rng, 1, 128)
        max_q = 1 if kind == "decode" else rng.randint(2, 8)
    # the plain form is padded: its scores stay below those of the largest listed case
    cap = min(32768, (1 << 31) // (n * max_q * kv_heads * group), (1 << 20) // n)
    cap = max(cap, max_q + 1)
    max_kv = _log(rng, max_q, cap)
    return dict(op="attend", dtype=dtype, requests=n, max_q=max_q, max_kv=max_kv, lens=rng.randint(0, 10**6),
                q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, page=page,
                window=rng.choice([0, 0, 0, max(1, max_kv // 3)]))


def _lens(case):
    """(q_len, kv_len) of an attention case's requests: the first one has the largest of both."""
    rng = random.Random(case["lens"])
    q, kv = [case["max_q"]], [case["max_kv"]]
    for _ in range(case["requests"] - 1):
        n = rng.randint(1, case["max_q"])
        q.append(n)
        kv.append(rng.randint(n, case["max_kv"]))
    return q, kv


def _read_lens(case):
    rng = random.Random(case["lens"])
    n = [case["max_len"]] + [rng.randint(1, case["max_len"]) for _ in range(case["requests"] - 1)]
    return [rng.randint(0, 2 * case["page"]) for _ in n], n


def _draft_lens(case):
    rng = random.Random(case["lens"])
    return [case["max_draft"]] + [rng.randint(0, case["max_draft"]) for _ in range(case["requests"] - 1)]


# ----------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _cu(lens):
    return _i32([0] + np.cumsum(lens).tolist())


def _pool(case, g, pages):
    """A cache of [pages][heads][page][head_dim] with contents as a model leaves them."""
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    out = {}
    for n in ("k", "v"):
        if case["dtype"] == "bf16":
            x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
            x.normal_(generator=g)
            out[n], out[n + "_scale"] = x, None
        else:
            x = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
            x.normal_(std=120.0, generator=g)
            out[n] = x.clamp_(-448, 448).to(E4M3)
            out[n + "_scale"] = torch.randint(118, 123, shape[:3], generator=g, device=DEV, dtype=torch.uint8)
    return out


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


def _library():
    from moe_expert_dispatch_route_gb300 import binding

    return binding


def prepare(case, seed):
    g = _gen(seed)
    st = {"case": case}
    op = case["op"]
    if op == "write":
        T, H, D, page = case["tokens"], case["kv_heads"], case["head_dim"], case["page"]
        pages = -(-T // page) + 3
        # the projection's output holds q, k and v of a token side by side
        qkv = _randn(g, T, 6 * H, D) * torch.exp(_randn(g, T, 1, 1) * 0.5)
        qkv = qkv.to(torch.bfloat16)
        st.update(keys=qkv[:, 4 * H:5 * H], values=qkv[:, 5 * H:])
        st["slots"] = torch.randperm(pages * page, generator=g, device=DEV)[:T].contiguous()
        st.update(_pool(case, g, pages))
    elif op == "read":
        start, n = _read_lens(case)
        pages, table = _table([a + b for a, b in zip(start, n)], case["page"], g)
        st.update(_pool(case, g, pages))
        T = sum(n)
        st.update(table=table, start=_i32(start), cu=_cu(n), tokens=T)
        shape = (T, case["kv_heads"], case["head_dim"])
        st.update(k_out=torch.empty(shape, dtype=torch.bfloat16, device=DEV),
                  v_out=torch.empty(shape, dtype=torch.bfloat16, device=DEV))
    elif op == "attend":
        q, kv = _lens(case)
        pages, table = _table(kv, case["page"], g)
        st.update(_pool(case, g, pages))
        T, H, D = sum(q), case["q_heads"], case["head_dim"]
        st.update(q=_randn(g, T, H, D).to(torch.bfloat16), table=table, cu=_cu(q), kv_len=_i32(kv),
                  scale=1.0 / math.sqrt(D))
        st.update(o=torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV),
                  lse=torch.empty(T, H, dtype=torch.float32, device=DEV))
    else:
        n = _draft_lens(case)
        N, B, V = sum(n), case["requests"], case["vocab"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        cu = _cu(n)
        owner = torch.repeat_interleave(torch.arange(B, device=DEV), torch.tensor(n, device=DEV), output_size=N)
        row = torch.arange(N, device=DEV) + owner  # target row of each drafted token
        logits = _randn(g, N + B, V) * 2.5
        st["target"] = torch.softmax(logits, -1).to(dt)
        # the draft model's opinion: near the target's, not the same
        logits = logits[row] + _randn(g, N, V) * 0.7
        draft = torch.softmax(logits, -1)
        del logits
        u = torch.rand(N, generator=g, device=DEV)
        ids = torch.searchsorted(draft.double().cumsum(-1), u[:, None].double()).clamp(max=V - 1)
        st.update(draft=draft.to(dt), ids=ids[:, 0].to(torch.int32).contiguous(), cu=cu)
        st["uniform"] = torch.rand(N, generator=g, device=DEV)
        st["uniform_sample"] = torch.rand(B, generator=g, device=DEV)
        st.update(out_ids=torch.empty(B, case["max_draft"] + 1, dtype=torch.int32, device=DEV),
                  out_len=torch.empty(B, dtype=torch.int32, device=DEV))
    if own:
        lib = _library()
        st["lib"] = lib
        st["err"] = torch.zeros(1, dtype=torch.int32, device=DEV)
        if op != "verify":
            st["cache"] = lib.kv_cache(st["k"], st["v"], st["k_scale"], st["v_scale"])
        if op == "attend":
            size = lib.moe_attn_workspace_size(st["cache"], case["q_heads"])
            st["ws"] = torch.zeros(size, dtype=torch.uint8, device=DEV)
            st["args"] = lib.attn_args(st["q"], st["o"], st["cu"], st["kv_len"], st["table"], case["max_q"],
                                       case["max_kv"], scale=st["scale"], causal=True, window=case["window"],
                                       lse=st["lse"], workspace=st["ws"], err_flag=st["err"])
    return st


# ------------------------------------------------------------------------------ one pass
def run(state):
    return {"write": _write, "read": _read, "attend": _attend, "verify": _verify}[state["case"]["op"]](state)


def _contents(st):
    return [st["k"], st["v"]] + ([] if st["k_scale"] is None else [st["k_scale"], st["v_scale"]])


def _write(st):
    if own:
        st["lib"].moe_kv_write(st["cache"], st["keys"], st["values"], st["slots"], err_flag=st["err"])
        return _contents(st)
    page, at = st["slots"] // st["case"]["page"], st["slots"] % st["case"]["page"]
    for n, x in (("k", st["keys"]), ("v", st["values"])):
        if st["k_scale"] is None:
            st[n][page, :, at] = x
            continue
        x = x.float()
        frac, e = torch.frexp(x.abs().amax(-1))
        s = torch.where(frac > 0.875, e - 8, e - 9)
        s = torch.where(frac == 0, 0, s).clamp(-100, 119)
        codes = torch.ldexp(x, -s[..., None]).clamp(-448, 448).to(E4M3)
        st[n].view(torch.uint8)[page, :, at] = codes.view(torch.uint8)
        st[n + "_scale"][page, :, at] = (s + 127).to(torch.uint8)
    return _contents(st)


def _scaled(st, n, page, at):
    """Cached tokens as numbers: [..., heads, head_dim] in 32 bits."""
    if st["k_scale"] is None:
        return st[n][page, :, at].float()
    codes = st[n].view(torch.uint8)[page, :, at].view(E4M3).float()
    return torch.ldexp(codes, st[n + "_scale"][page, :, at].int()[..., None] - 127)


def _read(st):
    if own:
        st["lib"].moe_kv_read(st["cache"], st["table"], st["start"], st["cu"], st["k_out"], st["v_out"],
                              err_flag=st["err"])
        return [st["k_out"], st["v_out"]]
    row = torch.arange(st["tokens"], device=DEV, dtype=torch.int32)
    b = torch.searchsorted(st["cu"][1:], row, right=True)
    pos = st["start"][b] + row - st["cu"][b]
    page = st["table"][b, pos // st["case"]["page"]].long()
    at = (pos % st["case"]["page"]).long()
    return [_scaled(st, n, page, at).to(torch.bfloat16) for n in ("k", "v")]


def _attend(st):
    if own:
        st["lib"].moe_attn_paged(st["cache"], st["args"])
        return [st["o"], st["lse"]]
    c = st["case"]
    B, Q, K, H, G, D = c["requests"], c["max_q"], c["max_kv"], c["kv_heads"], c["q_heads"] // c["kv_heads"], c["head_dim"]
    # the requests padded to the longest: queries [B, heads, group * Q, D], keys [B, heads, K, D]
    i, j = torch.arange(Q, device=DEV), torch.arange(K, device=DEV)
    n = st["cu"][1:] - st["cu"][:-1]
    T = st["q"].shape[0]
    at = (st["cu"][:-1, None] + i[None]).clamp(max=T - 1)
    q = st["q"].float()[at].view(B, Q, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * Q, D)
    page = st["table"].long()[:, j // c["page"]]
    k = _scaled(st, "k", page, (j % c["page"])[None].expand(B, K))
    s = q @ k.permute(0, 2, 3, 1) * st["scale"]
    del k
    pos = (st["kv_len"] - n)[:, None] + i[None]
    seen = (j[None, None] <= pos[..., None]) & (j[None, None] < st["kv_len"][:, None, None])
    if c["window"]:
        seen &= j[None, None] > (pos - c["window"])[..., None]
    s = s.view(B, H, G, Q, K).masked_fill_(~seen[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    s = s.sub_(torch.where(m == -math.inf, 0.0, m)).exp_()
    total = s.sum(-1, keepdim=True)
    v = _scaled(st, "v", page, (j % c["page"])[None].expand(B, K))
    v = torch.where((j[None] < st["kv_len"][:, None])[..., None, None], v, 0.0)
    o = (s.view(B, H, G * Q, K) @ v.permute(0, 2, 1, 3)).view(B, H, G, Q, D)
    o = torch.where(total > 0, o / total, 0.0)
    lse = m[..., 0] + total[..., 0].log()
    # back to the packed rows
    row = torch.arange(T, device=DEV, dtype=torch.int32)
    b = torch.searchsorted(st["cu"][1:], row, right=True)
    t = (row - st["cu"][b]).long()
    return [o.permute(0, 3, 1, 2, 4)[b, t].reshape(T, H * G, D).to(torch.bfloat16),
            lse.permute(0, 3, 1, 2)[b, t].reshape(T, H * G)]


def _verify(st):
    if own:
        st["lib"].moe_draft_verify(st["target"], st["draft"], st["cu"], st["ids"], st["uniform"],
                                   st["uniform_sample"], st["out_ids"], st["out_len"], err_flag=st["err"])
        return [st["out_ids"], st["out_len"]]
    c = st["case"]
    B, M, V = c["requests"], c["max_draft"], c["vocab"]
    n = (st["cu"][1:] - st["cu"][:-1]).long()
    N = st["ids"].shape[0]
    slot = torch.arange(M, device=DEV)[None]
    at = (st["cu"][:-1, None].long() + slot).clamp(max=N - 1)
    row = st["cu"][:-1, None].long() + torch.arange(B, device=DEV)[:, None] + slot
    ids = st["ids"][at].long()
    p = st["target"][row.clamp(max=N + B - 1), ids].double()
    q = st["draft"][at, ids].double()
    # products of two 24-bit significands are exact in 64 bits
    kept = (st["uniform"][at].double() * q < p) & (slot < n[:, None])
    count = kept.int().cumprod(-1).sum(-1)
    # the token after them: from what the target has beyond the draft, or from the target
    p = st["target"][st["cu"][:-1].long() + torch.arange(B, device=DEV) + count].float()
    q = st["draft"][(st["cu"][:-1].long() + count).clamp(max=N - 1)].float()
    r = torch.where((count < n)[:, None], p - q, p).clamp(0, 1)
    total = torch.floor(r.double() * 2.0**40).long().cumsum(-1)
    whole = torch.floor(st["uniform_sample"].double() * 2.0**24).long()
    end = total[:, -1]
    want = whole * (end >> 24) + (whole * (end & 0xFFFFFF) >> 24)
    token = torch.searchsorted(total, want[:, None], right=True)[:, 0]
    slot = torch.arange(M + 1, device=DEV)[None]
    ids = torch.cat([ids, ids[:, :1]], 1)
    out = torch.where(slot < count[:, None], ids, torch.where(slot == count[:, None], token[:, None], -1))
    return [out.to(torch.int32), (count + 1).to(torch.int32)]


# ------------------------------------------------------------------------------- the work
def _pairs(q, kv, window):
    """(query, key) pairs that a request's causal mask leaves."""
    first = kv - q
    if not window:
        return q * first + q * (q + 1) // 2
    pos = np.arange(first, kv)
    return int(np.minimum(pos + 1, window).sum())


def work(case):
    op = case["op"]
    if op == "verify":
        el = 4 if case["dtype"] == "f32" else 2
        n = _draft_lens(case)
        # one row of the target a request; the draft's row too where a token is refused, which the data decides
        return {"bytes": case["requests"] * (case["vocab"] * el + 4 * (case["max_draft"] + 4)) + sum(n) * (2 * el + 8),
                "flops": 2 * case["requests"] * case["vocab"]}
    H, D = case["kv_heads"], case["head_dim"]
    row = 2 * H * (2 * D if case["dtype"] == "bf16" else D + 1)  # one token in the cache
    if op == "write":
        return {"bytes": case["tokens"] * (4 * H * D + row + 8), "flops": 4 * case["tokens"] * H * D}
    if op == "read":
        T = sum(_read_lens(case)[1])
        return {"bytes": T * (4 * H * D + row + 4 / case["page"]), "flops": 2 * T * H * D}
    q, kv = _lens(case)
    held = sum(min(b, a + case["window"] - 1) if case["window"] else b for a, b in zip(q, kv))
    return {"bytes": held * row + sum(q) * case["q_heads"] * (4 * D + 4),
            "flops": 4 * D * case["q_heads"] * sum(_pairs(a, b, case["window"]) for a, b in zip(q, kv))}


# ------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    page = case.get("page")
    if op == "verify":
        return None  # whole numbers: equal on both sides
    if op == "write":
        out = []
        for n, x in (("k", st["keys"]), ("v", st["values"])):
            pool = st[n].double().transpose(1, 2).flatten(0, 1)  # [slots][heads][head_dim]
            x = x.double()
            if st["k_scale"] is not None:
                top = x.abs().amax(-1, keepdim=True)
                s = torch.ceil(torch.log2(top / 448))
                s = torch.where(448 * torch.exp2(s - 1) >= top, s - 1, s)
                s = torch.where(448 * torch.exp2(s) < top, s + 1, s).clamp(-100, 119)
                x = x / torch.exp2(s)
                # nearest of the 8-bit numbers, ties to even: steps of 2^(e - 3), and 2^-9 below 2^-6
                step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0**-6))) - 3)
                x = (torch.round(x / step) * step).clamp(-448, 448)
            pool[st["slots"]] = x
            out.append(pool.view(-1, page, case["kv_heads"], case["head_dim"]).transpose(1, 2).contiguous())
        return out + ([] if st["k_scale"] is None else [None, None])

    def rows(n, pages):
        x = st[n][pages].double()
        if st["k_scale"] is not None:
            x = x * torch.exp2(st[n + "_scale"][pages].double() - 127)[..., None]
        return x.transpose(1, 2).flatten(0, 1)  # [tokens][heads][head_dim]

    if op == "read":
        start, lens = _read_lens(case)
        return [torch.cat([rows(n, st["table"][b, :-(-(a + m) // page)].long())[a:a + m]
                           for b, (a, m) in enumerate(zip(start, lens))]) for n in ("k", "v")]
    q_len, kv_len = _lens(case)
    H, G = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    o, lse, first = [], [], 0
    for b, (m, n) in enumerate(zip(q_len, kv_len)):
        pages = st["table"][b, :-(-n // page)].long()
        k, v = rows("k", pages)[:n], rows("v", pages)[:n]
        pos, j = torch.arange(n - m, n, device=DEV)[:, None], torch.arange(n, device=DEV)[None]
        hidden = j > pos
        if case["window"]:
            hidden |= pos - j >= case["window"]
        ob = torch.empty(m, case["q_heads"], case["head_dim"], dtype=torch.float64, device=DEV)
        lb = torch.empty(m, case["q_heads"], dtype=torch.float64, device=DEV)
        for h in range(H):
            x = st["q"][first:first + m, h * G:(h + 1) * G].double()
            w = torch.einsum("mgd,nd->gmn", x, k[:, h]) * st["scale"]
            w.masked_fill_(hidden, -math.inf)
            z = torch.logsumexp(w, -1)
            w.sub_(z[..., None]).exp_()
            ob[:, h * G:(h + 1) * G] = torch.einsum("gmn,nd->mgd", w, v[:, h])
            lb[:, h * G:(h + 1) * G] = z.T
        o.append(ob)
        lse.append(lb)
        first += m
    return [torch.cat(o), torch.cat(lse)]
