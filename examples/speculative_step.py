"""A serving loop around the MoE layer: paged cache, attention, experts, draft verification.

A small random-weight decoder (two layers by default; attention heads and experts shaped like the
``qwen3_decode`` workload) serves a few requests: their prompts go through as ragged chunks, then every
step verifies a few drafted tokens a request.  Per layer and step

    moe_kv_write    the new tokens' keys and values into the cache (bf16, or e4m3 with --cache e4m3)
    moe_attn_paged  attention of the new tokens over it
    moe_layer_dbo   router top-k, dispatch, experts, combine, on two overlapped ubatches

and per step ``moe_draft_verify``.  Norms, projections and the draft model are plain torch: they stand
for the program around the library.  (Positions are not encoded; a real model rotates q and k.)

    python examples/speculative_step.py [--steps 8] [--requests 4] [--cache bf16|e4m3]
"""
from __future__ import annotations

import argparse
import math
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_expert_dispatch_route_gb300 import binding as B  # noqa: E402
from moe_expert_dispatch_route_gb300 import synth  # noqa: E402
from moe_expert_dispatch_route_gb300 import workloads as W  # noqa: E402

DEV = "cuda"
Q_HEADS, KV_HEADS, HEAD_DIM, PAGE = 32, 4, 128, 64


def norm(x):
    return torch.nn.functional.rms_norm(x, (x.shape[-1],))


class Layer:
    def __init__(self, wl, cfg, pages, e4m3, g):
        rand = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.float32)
        H = wl.hidden
        self.wqkv = (rand(H, (Q_HEADS + 2 * KV_HEADS) * HEAD_DIM) * H**-0.5).to(torch.bfloat16)
        self.wo = (rand(Q_HEADS * HEAD_DIM, H) * (Q_HEADS * HEAD_DIM)**-0.5).to(torch.bfloat16)
        self.router = rand(H, wl.num_experts) * H**-0.5
        self.experts = synth.weights(wl.num_experts + wl.num_shared, H, wl.inter, wl.dtype, seed=wl.seed, device=DEV)
        self.pool = torch.zeros(2, pages, KV_HEADS, PAGE, HEAD_DIM, dtype=torch.bfloat16, device=DEV)
        scales = (None, None)
        if e4m3:
            self.pool = self.pool.to(torch.float8_e4m3fn)
            self.scales = torch.full((2, pages, KV_HEADS, PAGE), 127, dtype=torch.uint8, device=DEV)
            scales = (self.scales[0], self.scales[1])
        self.cache = B.kv_cache(self.pool[0], self.pool[1], *scales)


class Decoder:
    """The model and its requests' state; `forward` runs new tokens of every request at once."""

    def __init__(self, requests, max_len, layers=2, vocab=4096, cache="bf16", workload=W.QWEN3_DECODE, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.wl, self.cfg = workload, B.config_of(workload)
        self.vocab, self.g = vocab, g
        self.embed = torch.randn(vocab, workload.hidden, generator=g, device=DEV).to(torch.bfloat16)
        self.head = (torch.randn(workload.hidden, vocab, generator=g, device=DEV) * workload.hidden**-0.5).to(
            torch.bfloat16)
        per = -(-max_len // PAGE)
        self.table = torch.randperm(requests * per, generator=g, device=DEV).to(torch.int32).view(requests, per)
        self.len = torch.zeros(requests, dtype=torch.int32, device=DEV)  # cached tokens of each request
        self.max_len = max_len
        self.layers = [Layer(workload, self.cfg, requests * per, cache == "e4m3", g) for _ in range(layers)]
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.layer_err = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.attn_ws = torch.zeros(B.moe_attn_workspace_size(self.layers[0].cache, Q_HEADS), dtype=torch.uint8,
                                   device=DEV)
        self.handle = B.moe_dbo_create()
        self.comm = torch.cuda.Stream()

    def close(self):
        B.moe_dbo_destroy(self.handle)

    def forward(self, tokens, cu, max_new):
        """tokens int64 [T], packed by request (cu int32 [B+1]): the next tokens after the cached ones.
        Probabilities of the token after each, fp32 [T][vocab]; the tokens are in the cache, but
        self.len does not count them yet."""
        T, requests = tokens.shape[0], self.len.shape[0]
        row = torch.arange(T, device=DEV, dtype=torch.int32)
        b = torch.searchsorted(cu[1:], row, right=True)
        pos = self.len[b] + row - cu[b]
        slots = self.table[b, pos // PAGE].long() * PAGE + pos % PAGE
        kv_len = self.len + cu[1:] - cu[:-1]
        max_kv = self.max_len
        x = self.embed[tokens]
        for ly in self.layers:
            qkv = (norm(x) @ ly.wqkv).view(T, Q_HEADS + 2 * KV_HEADS, HEAD_DIM)
            B.moe_kv_write(ly.cache, qkv[:, Q_HEADS:Q_HEADS + KV_HEADS], qkv[:, Q_HEADS + KV_HEADS:], slots,
                           err_flag=self.err)
            o = torch.empty(T, Q_HEADS, HEAD_DIM, dtype=torch.bfloat16, device=DEV)
            B.moe_attn_paged(ly.cache, B.attn_args(qkv[:, :Q_HEADS], o, cu, kv_len, self.table, max_new, max_kv,
                                                   1 / math.sqrt(HEAD_DIM), workspace=self.attn_ws,
                                                   err_flag=self.err))
            x = x + o.view(T, -1) @ ly.wo
            h = norm(x)
            logits = h.float() @ ly.router
            y = torch.empty_like(x)
            ids = torch.empty(T, self.wl.top_k, dtype=torch.int32, device=DEV)
            w = torch.empty(T, self.wl.top_k, dtype=torch.float32, device=DEV)
            ws = torch.empty(B.moe_layer_workspace_size(self.cfg, T), dtype=torch.uint8, device=DEV)
            args = B.layer_args(logits, h, ly.experts, y, ids, w, ws, err_flag=self.layer_err)
            B.moe_layer_dbo(self.handle, self.cfg, args, T, compute=torch.cuda.current_stream(), comm=self.comm)
            x = x + y
        assert requests == cu.shape[0] - 1
        return torch.softmax((norm(x) @ self.head).float(), -1)

    def draft(self, last, n):
        """n tokens a request from a model that looks at the last token only: ids [B * n] and their
        distributions [B * n][vocab]."""
        ids, probs = [], []
        for _ in range(n):
            p = torch.softmax((norm(self.embed[last]) @ self.head).float(), -1)
            last = torch.multinomial(p, 1, generator=self.g)[:, 0]
            ids.append(last)
            probs.append(p)
        return torch.stack(ids, 1).reshape(-1), torch.stack(probs, 1).reshape(-1, self.vocab)

    def step(self, last, n):
        """One speculative step after the tokens `last` [B]: n drafts a request, verified in one pass.
        Kept and drawn tokens int32 [B][n + 1] (-1 past them) and their number [B]."""
        requests = last.shape[0]
        ids, q = self.draft(last, n)
        tokens = torch.cat([last[:, None], ids.view(requests, n)], 1).reshape(-1)
        cu = torch.arange(requests + 1, dtype=torch.int32, device=DEV) * (n + 1)
        p = self.forward(tokens, cu, n + 1)
        cu_draft = torch.arange(requests + 1, dtype=torch.int32, device=DEV) * n
        out = torch.empty(requests, n + 1, dtype=torch.int32, device=DEV)
        count = torch.empty(requests, dtype=torch.int32, device=DEV)
        u = torch.rand(requests * (n + 1), generator=self.g, device=DEV)
        B.moe_draft_verify(p, q, cu_draft, ids.to(torch.int32), u[:requests * n], u[requests * n:], out, count,
                           err_flag=self.err)
        self.len += count  # the refused drafts' slots are written again by the next step
        return out, count


def serve(requests=4, steps=8, drafts=4, prompt=300, cache="bf16", seed=0, **kw):
    """Prompts of ragged lengths, then `steps` speculative steps; returns the tokens of each request."""
    m = Decoder(requests, prompt + (steps + 1) * (drafts + 1), cache=cache, seed=seed, **kw)
    lens = [max(1, prompt - 37 * i) for i in range(requests)]
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    tokens = torch.randint(0, m.vocab, (sum(lens),), generator=m.g, device=DEV)
    p = m.forward(tokens, cu, max(lens))
    m.len += cu[1:] - cu[:-1]
    last = p[cu[1:].long() - 1].argmax(-1)
    made = [[t] for t in last.tolist()]
    t0, total = time.perf_counter(), 0
    for _ in range(steps):
        out, count = m.step(last, drafts)
        last = out.gather(1, count[:, None].long() - 1)[:, 0].long()
        for r, (row, n) in enumerate(zip(out.tolist(), count.tolist())):
            made[r] += row[:n]
            total += n
    seconds = time.perf_counter() - t0
    err = (int(m.err.item()), int(m.layer_err.item()))
    m.close()
    if err != (0, 0):
        raise RuntimeError(f"a kernel reported {err}")
    return made, total / seconds


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--requests", type=int, default=4)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=300)
    ap.add_argument("--cache", choices=["bf16", "e4m3"], default="bf16")
    a = ap.parse_args()
    made, rate = serve(a.requests, a.steps, a.drafts, a.prompt, a.cache)
    for r, t in enumerate(made):
        print(f"request {r}: {len(t)} tokens: {t[:12]}{' ...' if len(t) > 12 else ''}")
    print(f"{rate:.0f} tokens/s with the host reading every step's tokens")


if __name__ == "__main__":
    main()
