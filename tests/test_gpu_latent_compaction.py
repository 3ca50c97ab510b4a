"""examples/latent_step.py: what a step keeps of its trees, with the target's choices set by hand so that every branch is
taken, and a tree's nodes against their branches fed as chains, with the routing fixed so that no tie can excuse one."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu
DEV = "cuda"
# nodes that the target agrees with, from the root, in a tree whose parents are [-1, 0, 0, 0, 1, 1, 4]
PATHS = [[0], [0, 1], [0, 2], [0, 3], [0, 1, 4], [0, 1, 5], [0, 1, 4, 6]]


@pytest.mark.parametrize("before", [0, 60, 63])
def test_the_kept_branch_moves_to_its_place(before):
    """Rows of the branch's nodes are, bit for bit, where a chain's would be; no other row changes."""
    import latent_step as S

    requests, nodes = len(PATHS), len(S.PARENT)
    m = S.Decoder(requests, 128)
    g = torch.Generator(device=DEV).manual_seed(1)
    for ly in m.layers:
        ly.pool.normal_(generator=g)
    m.len += before
    ids = torch.randperm(m.vocab, generator=g, device=DEV)[:requests * nodes].view(requests, nodes)
    m.draft = lambda last: ids
    after = torch.randperm(m.vocab, generator=g, device=DEV)
    after = after[~torch.isin(after, ids)][:requests]  # the target's last choices: in no draft
    real, seen = m.forward, {}

    def forward(tokens, cu, max_new, **kw):
        p = real(tokens, cu, max_new, **kw).view(requests, nodes, -1)
        for b, path in enumerate(PATHS):
            for node, child in zip(path, path[1:] + [None]):
                p[b, node, after[b] if child is None else ids[b, child]] = 2.0  # the largest
        seen["pools"] = [ly.pool.clone() for ly in m.layers]
        return p.view(requests * nodes, -1)

    m.forward = forward
    out, count = m.step(ids[:, 0])
    assert int(m.err.item()) == 0 and count.tolist() == [len(p) for p in PATHS]
    assert m.len.tolist() == [before + len(p) for p in PATHS]
    for b, path in enumerate(PATHS):
        want = [int(ids[b, n]) for n in path[1:]] + [int(after[b])]
        assert out[b].tolist() == want + [-1] * (out.shape[1] - len(want))
    at = m.slots(torch.arange(requests, device=DEV)[:, None], before + torch.arange(nodes, device=DEV)[None].expand(requests, -1))
    for ly, old in zip(m.layers, seen["pools"]):
        old = old.view(-1, old.shape[2])
        want = old.clone()
        for b, path in enumerate(PATHS):
            want[at[b, :len(path)]] = old[at[b, path]]
        assert torch.equal(want, ly.pool.view_as(want))
    m.close()


@pytest.mark.parametrize("prompt", [5, 70])
def test_every_node_is_its_chain(prompt):
    """Two layers round activations at different places (bf16: 2^-8 of one each); with the experts' choice fixed (equal
    logits: the first ones), probabilities are off by a few such roundings of the logits, whose spread is about 1."""
    import latent_step as S

    g = torch.Generator(device=DEV).manual_seed(prompt)
    first, ids = (torch.randint(0, 4096, (n,), generator=g, device=DEV) for n in (prompt, len(S.PARENT)))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    m = S.Decoder(1, 128)
    for ly in m.layers:
        ly.router.zero_()
    m.forward(first, i32(0, prompt), prompt, prompt=True)
    m.len += prompt
    got = m.forward(ids, i32(0, len(ids)), len(ids), tree=torch.tensor(S.BRANCH, device=DEV))
    for i, bits in enumerate(S.BRANCH):
        chain = ids[[j for j in range(len(ids)) if bits >> j & 1]]
        want = m.forward(chain, i32(0, len(chain)), len(chain))[-1]
        others = [0.5 * (want - got[j]).abs().sum().item() for j in range(len(ids)) if j != i]
        off = 0.5 * (want - got[i]).abs().sum().item()
        assert off < 0.03 and min(others) > 0.1, (i, off, others)  # and is told from every other node
    assert int(m.err.item()) == 0
    m.close()
