"""Latent attention, trees and block norms together, as a serving program calls them (examples/latent_step.py)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_loop_runs():
    import latent_step as S

    made, _ = S.serve(requests=3, steps=4, prompt=200)
    assert all(1 + 4 <= len(t) <= 1 + 4 * 4 for t in made)
    assert all(0 <= x < 4096 for t in made for x in t)
    again, _ = S.serve(requests=3, steps=4, prompt=200)
    assert made == again


def test_both_forms_give_the_same_probabilities():
    """The same tokens as one prompt (expanded form), as chunks over the cache (absorbed), and their last ones as a tree
    that is a chain.  The paths round at different places: keys and values, or queries and outputs, once more to bf16,
    2^-8 of an activation in each of two layers; total variation 3 % is ten such roundings of the logits, whose spread
    is about 1."""
    import latent_step as S

    tokens = torch.randint(0, 4096, (2 * 90,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    cut = lambda n: torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    m = S.Decoder(2, 128)
    whole = m.forward(tokens, cut(90), 90, prompt=True).view(2, 90, -1)
    m.close()
    m = S.Decoder(2, 128)
    at, parts = 0, []
    for n, how in ((50, "prompt"), (1, ""), (5, ""), (33, ""), (1, "tree")):
        tree = torch.tensor([(1 << (i + 1)) - 1 for i in range(n)] * 2, device="cuda") if how == "tree" else None
        x = tokens.view(2, 90)[:, at:at + n].reshape(-1)
        parts.append(m.forward(x, cut(n), n, prompt=how == "prompt", tree=tree).view(2, n, -1))
        m.len += n
        at += n
    assert int(m.err.item()) == 0 and int(m.layer_err.item()) == 0
    m.close()
    tv = 0.5 * (whole - torch.cat(parts, 1)).abs().sum(-1)
    # a router near a tie may pick another expert on one path: that token's output is another one
    assert tv.median() < 0.03 and (tv < 0.03).float().mean() > 0.8, (tv.median().item(), tv.max().item())


def test_a_tree_node_is_its_chain():
    """Each node's probabilities are those of its branch fed as a chain."""
    import latent_step as S

    g = torch.Generator(device="cuda").manual_seed(5)
    prompt, ids = (torch.randint(0, 4096, (n,), generator=g, device="cuda") for n in (70, len(S.PARENT)))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    m = S.Decoder(1, 128)
    m.forward(prompt, i32(0, 70), 70, prompt=True)
    m.len += 70
    got = m.forward(ids, i32(0, len(ids)), len(ids), tree=torch.tensor(S.BRANCH, device="cuda"))
    off = []
    for i, bits in enumerate(S.BRANCH):
        chain = ids[[j for j in range(len(ids)) if bits >> j & 1]]
        want = m.forward(chain, i32(0, len(chain)), len(chain))[-1]
        off.append(0.5 * (want - got[i]).abs().sum().item())
    assert int(m.err.item()) == 0
    m.close()
    # as above; the same kernels on other rows of a tile
    assert sorted(off)[len(off) // 2] < 0.03, off


def test_a_perfect_tree_is_kept():
    """A draft whose first guesses are the target's own choices: the deepest branch is kept whole every step, and the
    cache then holds it where a chain's tokens would be."""
    import latent_step as S

    m = S.Decoder(2, 64)
    last = torch.tensor([1, 2], device="cuda")
    cu = lambda n: torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")

    def draft(last):
        deep = [last]
        for _ in range(3):  # the chain that the target would choose
            x = torch.stack(deep, 1)
            n = x.shape[1]
            deep.append(m.forward(x.reshape(-1), cu(n), n).view(2, n, -1)[:, -1].argmax(-1))
        other = (deep[1] + 1) % 4096
        return torch.stack([last, deep[1], other, other, deep[2], (deep[2] + 1) % 4096, deep[3]], 1)

    m.draft = draft
    out, count = m.step(last)
    assert int(m.err.item()) == 0
    # (a near tie may be decided otherwise by the tree's kernel: at least the first choice is kept)
    assert all(c >= 2 for c in count.tolist())
    if count.tolist() == [4, 4]:
        chain = torch.cat([last[:, None], out[:, :3]], 1)
        rows = torch.stack([ly.pool.view(-1, 576)[m.slots(torch.tensor([[0], [1]], device="cuda"),
                                                          torch.arange(4, device="cuda")[None].expand(2, 4))]
                            for ly in m.layers])
        m.len -= 4
        m.forward(chain.reshape(-1), cu(4), 4)
        again = torch.stack([ly.pool.view(-1, 576)[m.slots(torch.tensor([[0], [1]], device="cuda"),
                                                           torch.arange(4, device="cuda")[None].expand(2, 4))]
                             for ly in m.layers])
        assert (rows.float() - again.float()).abs().median().item() < 0.05
    m.close()
