"""The serving operators together, as a serving program calls them (examples/speculative_step.py)."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_loop_runs(cache):
    import speculative_step as S

    made, _ = S.serve(requests=3, steps=4, drafts=3, prompt=200, cache=cache)
    assert all(1 + 4 <= len(t) <= 1 + 4 * 4 for t in made)
    assert all(0 <= x < 4096 for t in made for x in t)
    again, _ = S.serve(requests=3, steps=4, drafts=3, prompt=200, cache=cache)
    assert made == again


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_cached_steps_agree_with_one_pass(cache):
    """The same tokens fed as one prompt chunk, or a few at a time over the cache (other kernels,
    other splits), give the same probabilities.  The two paths round activations to bf16 at the
    same places, and differ by the rounding of attention's probabilities and by the order of fp32
    sums: 2^-8 of an activation in each of two layers of residual sums.  Total variation 3 % is
    ten such roundings of the logits, whose spread is about 1."""
    import speculative_step as S

    tokens = torch.randint(0, 4096, (2 * 90,), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    cut = lambda n: torch.tensor([0, n, 2 * n], dtype=torch.int32, device="cuda")
    m = S.Decoder(2, 128, cache=cache)
    whole = m.forward(tokens, cut(90), 90).view(2, 90, -1)
    m.close()
    m = S.Decoder(2, 128, cache=cache)
    at = 0
    parts = []
    for n in (50, 1, 5, 33, 1):
        parts.append(m.forward(tokens.view(2, 90)[:, at:at + n].reshape(-1), cut(n), n).view(2, n, -1))
        m.len += n
        at += n
    m.close()
    tv = 0.5 * (whole - torch.cat(parts, 1)).abs().sum(-1)
    # a router near a tie may pick another expert on one path: that token's output is another one
    assert tv.median() < 0.03 and (tv < 0.03).float().mean() > 0.8, (tv.median().item(), tv.max().item())


def test_a_perfect_draft_is_kept():
    """A draft model that is the target: every token is kept (u q < p with u below 1)."""
    import speculative_step as S

    m = S.Decoder(2, 64)
    last = torch.tensor([1, 2], device="cuda")

    def draft(_, n):
        ids, probs, seen = [], [], [last]
        for _ in range(n):
            k = len(seen)
            cu = torch.tensor([0, k, 2 * k], dtype=torch.int32, device="cuda")
            p = m.forward(torch.stack(seen, 1).reshape(-1), cu, k).view(2, k, -1)[:, -1]
            seen.append(torch.multinomial(p, 1, generator=m.g)[:, 0])
            ids.append(seen[-1])
            probs.append(p)
        return torch.stack(ids, 1).reshape(-1), torch.stack(probs, 1).reshape(-1, m.vocab)

    m.draft = draft
    real = S.B.moe_draft_verify

    def exact(p, q, *a, **kw):  # the pass over all drafts rounds differently: give it the draft's numbers
        p = p.clone().view(2, 4, -1)
        p[:, :3] = q.view(2, 3, -1)
        real(p.view(8, -1), q, *a, **kw)

    S.B.moe_draft_verify = exact
    try:
        out, count = m.step(last, 3)
    finally:
        S.B.moe_draft_verify = real
        m.close()
    assert count.tolist() == [4, 4] and (out >= 0).all()
