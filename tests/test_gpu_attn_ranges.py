"""Attention over an e4m3 cache whose scales lie far apart: a row's output goes by the keys that it sees
and by their weights, not by the largest scale that stands beside them."""
import pytest

from test_gpu_attn import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 6, 70])
@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
def test_a_scale_near_the_smallest(n, dtype):
    """All scores 0 or next to it: the masked ones must not become -inf * 0."""
    for scale in (2.0**-60, 2.0**-126):
        c = Case([n, n], [200, 90], dtype=dtype, scale=scale)
        c.q = c.q * 0
        c.qd.zero_()
        c.check()
