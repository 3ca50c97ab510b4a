"""The bounds of exact_ref tell a right answer from wrong ones for every kind of input that the GPU tests use."""
import numpy as np
import pytest
import torch

import exact_ref as X
import latent_ref as R


def bf16(x):
    return torch.tensor(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("kind", list(X.LATENT))
@pytest.mark.parametrize("width,values", [(576, 512), (192, 128), (128, 128), (64, 64)])
@pytest.mark.parametrize("n,kv", [(1, 700), (6, 1300)])
def test_wrong_answers_are_refused(kind, width, values, n, kv):
    q, k, v, scale = X.latent_numbers(np.random.default_rng(kv + n), kind, n, 3, kv, width, values)
    seen = R.chain(n, kv)
    ref = X.attention(q, k, v, seen, scale)
    o, lse = ref[0], ref[1]
    X.check(bf16(o), lse.astype(np.float32).astype(np.float64), ref, "the answer")
    # what a kernel may do: probabilities rounded to bf16, their sum taken before
    s = np.where(seen[:, None], np.einsum("nhd,kd->nhk", q, k) * scale, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    X.check(bf16(np.einsum("nhk,kd->nhd", bf16(p), v) / p.sum(-1, keepdims=True)), lse, ref, "rounded probabilities")
    wrong = {"zero": 0 * o, "negative": -o, "one and a half": 1.5 * o, "the next row's": np.roll(o, 1, axis=1)}
    if kind != "flat":  # (averages of many values of either sign: their roundings are a tenth of them)
        wrong["one part in 30"] = o * (1 + 1 / 30)
    late = np.where(np.arange(kv) < kv - kv // 8, s, -np.inf)  # the last keys forgotten
    if kind not in ("falling", "rise and fall"):  # (they weigh nothing there)
        e = np.exp(late - late.max(-1, keepdims=True))
        wrong["keys forgotten"] = np.einsum("nhk,kd->nhd", e / e.sum(-1, keepdims=True), v)
    for what, x in wrong.items():
        with pytest.raises(AssertionError):
            X.check(x, lse, ref, what)
    for off in (0.01 + np.abs(lse) * 1e-3, -0.01 - np.abs(lse) * 1e-3):
        with pytest.raises(AssertionError):
            X.check(o, lse + off, ref, "lse")


def test_a_bound_that_says_nothing_is_refused():
    o = np.zeros((1, 1, 4))
    with pytest.raises(AssertionError, match="says nothing"):
        X.check(o, np.zeros((1, 1)), (o, np.zeros((1, 1)), o, np.full((1, 1), 0.1)), "")
    with pytest.raises(AssertionError):  # scores that fp32 rounds
        X.attention(np.full((1, 1, 64), 0.3), np.ones((2, 64)), np.ones((2, 8)), np.ones((1, 2), dtype=bool), 1.0)
