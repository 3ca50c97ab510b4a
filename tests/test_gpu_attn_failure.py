"""A CTA of the attention that gives up: what the other CTAs and the next call on its workspace see of it."""
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [5000]), ([2, 1], [3000, 40]), ([100], [9000]), ([150, 40], [700, 6000])])
@pytest.mark.parametrize("max_ctas", [0, 5])
def test_the_workspace_after_a_timeout(dtype, q_lens, kv_lens, max_ctas):
    """Parts of query tiles that the first CTA does not deliver are counted all the same: the call reports the
    timeout and leaves its counters zero, and the next one on the same workspace is right."""
    c = Case(q_lens, kv_lens, Hq=8, H=2, dtype=dtype, page=64)
    for _ in range(2):
        B.moe_debug_inject_wait(True, 1000000)
        try:
            c.run(max_ctas=max_ctas)
        finally:
            B.moe_debug_inject_wait(False)
        assert int(c.err.item()) == 8
        assert int(c.ws[:4096].count_nonzero().item()) == 0, "the counters are left zero"
        c.err.zero_()
        c.check(max_ctas=max_ctas)
