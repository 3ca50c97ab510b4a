"""A serving loop with latent attention around the MoE layer: trees of drafted tokens, verified in one pass.

A small random-weight decoder (two layers by default, shaped like the ``dsv2lite`` workload) keeps one latent
vector and one rotary key a token.  Prompts go through in the expanded form of the attention; then every step
drafts a tree of tokens a request, runs it through the absorbed form, keeps the branch that the target would have
chosen and moves its cached rows to where a chain's would be.  Per layer and step

    moe_block_norm     the residual sum before each block and the norm of its input
    moe_latent_write   the new tokens' latent vectors, normed, into the pages of the cache
    moe_attn_expanded  attention of a prompt, keys and values of every head written out
    moe_attn_latent    attention of a tree over the cache
    moe_layer_dbo      the experts

Projections, the draft model and the choice of the branch are plain torch: they stand for the program around the
library.  (Positions are not encoded; a real model rotates the last 64 numbers of q and the rotary keys.)

    python examples/latent_step.py [--steps 8] [--requests 4] [--prompt 300]
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from moe_expert_dispatch_route_gb300 import binding as B  # noqa: E402
from moe_expert_dispatch_route_gb300 import synth  # noqa: E402
from moe_expert_dispatch_route_gb300 import workloads as W  # noqa: E402

DEV = "cuda"
HEADS, PAGE, SCALE = 12, 64, (B.HEAD + B.ROPE)**-0.5
BF16 = torch.bfloat16

# A tree of drafted tokens: node 0 is the token before them, node i the RANK[i]-th best guess after its parent.
PARENT = [-1, 0, 0, 0, 1, 1, 4]
RANK = [0, 0, 1, 2, 0, 1, 0]
BRANCH = []
for _i, _p in enumerate(PARENT):
    BRANCH.append((BRANCH[_p] if _p >= 0 else 0) | 1 << _i)


class Layer:
    def __init__(self, wl, pages, g):
        rand = lambda *s: torch.randn(*s, generator=g, device=DEV) * s[-2]**-0.5
        H = wl.hidden
        self.wq, self.wdown = rand(H, HEADS * (B.HEAD + B.ROPE)).to(BF16), rand(H, B.LATENT + B.ROPE).to(BF16)
        self.wuk, self.wuv = rand(HEADS, B.LATENT, B.HEAD).to(BF16), rand(HEADS, B.LATENT, B.HEAD).to(BF16)
        self.wo = rand(HEADS * B.HEAD, H).to(BF16)
        self.router = rand(H, wl.num_experts)
        self.norms = [(1 + 0.1 * torch.randn(n, generator=g, device=DEV)).to(BF16) for n in (H, B.LATENT, H)]
        self.experts = synth.weights(wl.num_experts + wl.num_shared, H, wl.inter, wl.dtype, seed=wl.seed, device=DEV)
        self.pool = torch.zeros(pages, PAGE, B.LATENT + B.ROPE, dtype=BF16, device=DEV)
        self.cache = B.latent_cache(self.pool)


class Decoder:
    """The model and its requests' state; `forward` runs new tokens of every request at once."""

    def __init__(self, requests, max_len, layers=2, vocab=4096, workload=W.DSV2LITE, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.wl, self.cfg, self.vocab, self.g, self.max_len = workload, B.config_of(workload), vocab, g, max_len
        self.embed = torch.randn(vocab, workload.hidden, generator=g, device=DEV).to(BF16)
        self.head = (torch.randn(workload.hidden, vocab, generator=g, device=DEV) * workload.hidden**-0.5).to(BF16)
        self.last_norm = torch.ones(workload.hidden, dtype=BF16, device=DEV)
        per = -(-max_len // PAGE)
        self.table = torch.randperm(requests * per, generator=g, device=DEV).to(torch.int32).view(requests, per)
        self.len = torch.zeros(requests, dtype=torch.int32, device=DEV)  # cached tokens of each request
        self.layers = [Layer(workload, requests * per, g) for _ in range(layers)]
        self.err, self.layer_err = torch.zeros(2, 1, dtype=torch.int32, device=DEV)
        size = max(B.moe_attn_latent_workspace_size(self.layers[0].cache, HEADS), B.moe_attn_expanded_workspace_size(HEADS))
        self.ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
        self.handle = B.moe_dbo_create()
        self.comm = torch.cuda.Stream()

    def close(self):
        B.moe_dbo_destroy(self.handle)

    def slots(self, b, pos):
        """Places in the pool of positions `pos` of requests `b`."""
        return self.table[b, pos // PAGE].long() * PAGE + pos % PAGE

    def forward(self, tokens, cu, max_new, prompt=False, tree=None):
        """tokens int64 [T], packed by request (cu int32 [B+1]): the next tokens after the cached ones, or (tree
        int64 [T]) trees of them.  A prompt has none before it.  Probabilities of the token after each, fp32
        [T][vocab]; the tokens are in the cache, but self.len does not count them yet."""
        T = tokens.shape[0]
        row = torch.arange(T, device=DEV, dtype=torch.int32)
        b = torch.searchsorted(cu[1:], row, right=True)
        slots = self.slots(b, self.len[b] + row - cu[b])
        kv_len = self.len + cu[1:] - cu[:-1]
        x = self.embed[tokens].float()  # the residual is kept in 32 bits
        y = torch.zeros(T, self.wl.hidden, dtype=BF16, device=DEV)
        h = torch.empty_like(y)
        for ly in self.layers:
            before, latent, after = ly.norms
            B.moe_block_norm(y, h, before, resid=x, resid_out=x)
            q = (h @ ly.wq).view(T, HEADS, B.HEAD + B.ROPE)
            down = h @ ly.wdown
            B.moe_latent_write(ly.cache, down[:, :B.LATENT], down[:, B.LATENT:], slots, weight=latent, err_flag=self.err)
            if prompt:
                c = ly.pool.view(-1, B.LATENT + B.ROPE)[slots]
                k, v = (torch.einsum("tl,hld->thd", c[:, :B.LATENT], w) for w in (ly.wuk, ly.wuv))
                o = torch.empty(T, HEADS, B.HEAD, dtype=BF16, device=DEV)
                B.moe_attn_expanded(B.attn_expanded_args(q, k, c[:, B.LATENT:], v, o, cu, cu, max_new, max_new, SCALE,
                                                         workspace=self.ws, err_flag=self.err))
            else:
                qa = torch.cat([torch.einsum("thd,hld->thl", q[..., :B.HEAD], ly.wuk), q[..., B.HEAD:]], 2)
                ol = torch.empty(T, HEADS, B.LATENT, dtype=BF16, device=DEV)
                args = B.attn_latent_args(qa, ol, cu, kv_len, self.table, max_new, self.max_len, SCALE, workspace=self.ws,
                                          err_flag=self.err)
                B.moe_attn_latent(ly.cache, args, tree=tree)
                o = torch.einsum("thl,hld->thd", ol, ly.wuv)
            B.moe_block_norm(o.reshape(T, -1) @ ly.wo, h, after, resid=x, resid_out=x)
            ids = torch.empty(T, self.wl.top_k, dtype=torch.int32, device=DEV)
            w = torch.empty(T, self.wl.top_k, dtype=torch.float32, device=DEV)
            ws = torch.empty(B.moe_layer_workspace_size(self.cfg, T), dtype=torch.uint8, device=DEV)
            args = B.layer_args(h.float() @ ly.router, h, ly.experts, y, ids, w, ws, err_flag=self.layer_err)
            B.moe_layer_dbo(self.handle, self.cfg, args, T, compute=torch.cuda.current_stream(), comm=self.comm)
        B.moe_block_norm(y, h, self.last_norm, resid=x)
        return torch.softmax((h @ self.head).float(), -1)

    def draft(self, last):
        """A tree of tokens after each of `last` [B], from a model that looks at the token before alone: [B][nodes]."""
        nodes = [last]
        for parent, rank in zip(PARENT[1:], RANK[1:]):
            guess = (torch.nn.functional.rms_norm(self.embed[nodes[parent]].float(), (self.wl.hidden,)).to(BF16) @ self.head)
            nodes.append(guess.topk(rank + 1).indices[:, rank])
        return torch.stack(nodes, 1)

    def step(self, last):
        """One step after the tokens `last` [B]: the tokens that the target chooses along its branch of the tree, and
        the one after them, int64 [B][depth + 1] (-1 past them), and their number [B]."""
        requests, nodes = last.shape[0], len(PARENT)
        ids = self.draft(last)
        cu = torch.arange(requests + 1, dtype=torch.int32, device=DEV) * nodes
        tree = torch.tensor(BRANCH, device=DEV).repeat(requests)
        best = self.forward(ids.reshape(-1), cu, nodes, tree=tree).argmax(-1).view(requests, nodes)
        # down the branch that the target agrees with
        at = torch.zeros(requests, dtype=torch.int64, device=DEV)
        parent = torch.tensor(PARENT, device=DEV)
        path, out, alive = [at], [best[:, 0]], torch.ones(requests, dtype=torch.bool, device=DEV)
        for _ in range(max(bin(x).count("1") for x in BRANCH) - 1):
            fits = (parent[None] == at[:, None]) & (ids == out[-1].clamp(min=0)[:, None]) & alive[:, None]
            alive = fits.any(1)
            at = torch.where(alive, fits.int().argmax(1), at)
            path.append(at)
            out.append(torch.where(alive, best.gather(1, at[:, None])[:, 0], -1))
        out, path = torch.stack(out, 1), torch.stack(path, 1)
        count = (out >= 0).sum(1).to(torch.int32)
        # the branch's rows of the cache to where a chain's would be (in its order, no row lies before its place)
        b = torch.arange(requests, device=DEV)
        for i in range(1, path.shape[1]):
            keep = i < count
            src, dst = self.slots(b, self.len + path[:, i]), self.slots(b, self.len + i)
            for ly in self.layers:
                flat = ly.pool.view(-1, B.LATENT + B.ROPE)
                flat[dst] = torch.where(keep[:, None], flat[src], flat[dst])
        self.len += count
        return out, count


def serve(requests=4, steps=8, prompt=300, seed=0, **kw):
    """Prompts of ragged lengths, then `steps` steps; returns the tokens of each request."""
    m = Decoder(requests, prompt + (steps + 1) * len(PARENT), seed=seed, **kw)
    lens = [max(1, prompt - 37 * i) for i in range(requests)]
    cu = torch.tensor([0] + torch.tensor(lens).cumsum(0).tolist(), dtype=torch.int32, device=DEV)
    tokens = torch.randint(0, m.vocab, (sum(lens),), generator=m.g, device=DEV)
    last = m.forward(tokens, cu, max(lens), prompt=True)[cu[1:].long() - 1].argmax(-1)
    m.len += cu[1:] - cu[:-1]
    made = [[t] for t in last.tolist()]
    t0, total = time.perf_counter(), 0
    for _ in range(steps):
        out, count = m.step(last)
        last = out.gather(1, count[:, None].long() - 1)[:, 0]
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
    ap.add_argument("--prompt", type=int, default=300)
    a = ap.parse_args()
    made, rate = serve(a.requests, a.steps, a.prompt)
    for r, t in enumerate(made):
        print(f"request {r}: {len(t)} tokens: {t[:12]}{' ...' if len(t) > 12 else ''}")
    print(f"{rate:.0f} tokens/s with the host reading every step's tokens")


if __name__ == "__main__":
    main()
