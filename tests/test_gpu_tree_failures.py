"""moe_attn_tree where something is amiss: bad lengths and pages, waits that run out, rows that are nobody's."""
import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu
KERNELS = [([3, 2], (8, 2)), ([40, 30], (8, 2))]  # few rows a key/value head, and tiles


@pytest.mark.parametrize("q_lens,heads", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_bad_lengths_and_pages(q_lens, heads, dtype):
    n, T = q_lens[0], sum(q_lens)
    c = Case(q_lens, [300, 200], *heads, dtype=dtype)
    want = c.run()[0].copy()
    c.kv[0] = 5000
    o, _ = c.run()
    assert int(c.err.item()) == 7 and np.all(o[:n] == 77.0) and np.array_equal(o[n:], want[n:])
    for bad in (10**6, -1):
        c = Case(q_lens, [300, 200], *heads, dtype=dtype)
        c.table[1, 0] = bad  # its tokens read as zeros
        o, _ = c.run()
        assert int(c.err.item()) == 7 and np.array_equal(o[:n], want[:n]) and np.isfinite(o[n:]).all()
    c = Case(q_lens, [300, 200], *heads, dtype=dtype)
    c.cu[2] = n  # the second request's rows are nobody's
    o, lse = c.run()
    assert int(c.err.item()) == 0 and np.array_equal(o[:n], want[:n]) and np.all(o[n:T] == 77.0) and np.all(lse[n:T] == 77.0)


@pytest.mark.parametrize("q_lens,heads", KERNELS)
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_first_cta_gives_up(q_lens, heads, dtype):
    c = Case(q_lens, [3000, 500], *heads, dtype=dtype)
    want = c.run()[0].copy()
    B.moe_debug_inject_wait(True, 2_000_000)
    try:
        c.run()
    finally:
        B.moe_debug_inject_wait(False)
    assert int(c.err.item()) == 8 and int(c.ws[:4096].count_nonzero().item()) == 0
    c.err.zero_()
    assert np.array_equal(c.run()[0], want) and int(c.err.item()) == 0
