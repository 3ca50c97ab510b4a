"""moe_block_norm where something is amiss: a bounded wait that runs out, infinities and NaN among the numbers."""
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"
TIMEOUT = 8


def tensors(T, H, dtype, resid, gate, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    rand = lambda *s, t=dtype: torch.randn(*s, generator=g, device=DEV).to(t)
    return dict(y=rand(T, H), resid=rand(T, H, t=resid), pre_weight=rand(H), post_weight=rand(H),
                gate=None if gate == 0 else rand(1 if gate == 1 else T, H))


def run(t, inplace=False, out=True, **kw):
    """(resid_out, out) of copies of the tensors."""
    y, resid = t["y"].clone(), t["resid"].clone()
    ro = resid if inplace else torch.full_like(resid, 7)
    o = None if not out else y if inplace else torch.full_like(y, 7)
    B.moe_block_norm(y, o, t["pre_weight"] if out else None, resid=resid, resid_out=ro, post_weight=t["post_weight"],
                     gate=t["gate"], **kw)
    torch.cuda.synchronize()
    return ro, o


@pytest.mark.parametrize("dtype,resid", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float32, torch.float32)])
@pytest.mark.parametrize("H", [1032, 2048, 2304, 7168, 8192])
@pytest.mark.parametrize("T,max_ctas,inplace,out", [(29, 2, False, True), (29, 1, True, True), (3, 2, False, False), (400, 0, True, True)])
def test_a_wait_that_runs_out(H, dtype, resid, T, max_ctas, inplace, out):
    """The first CTA's copies are on their way when it gives up: its rows are NaN, the other CTAs' are right, the error is
    told, and the next call is as good as any."""
    t = tensors(T, H, dtype, resid, 2 if H == 2048 else 1)
    assert B.moe_comm_error(clear=True) == 0
    want = run(t, inplace, out, max_ctas=max_ctas)
    B.moe_debug_inject_wait(True, 2_000_000)
    try:
        got = run(t, inplace, out, max_ctas=max_ctas)
    finally:
        B.moe_debug_inject_wait(False)
    assert B.moe_comm_error() == TIMEOUT and B.moe_comm_error(clear=True) == TIMEOUT and B.moe_comm_error() == 0
    for a, b in zip(want, got):
        if a is None:
            continue
        void = b.isnan().any(1)
        assert torch.equal(void, b.isnan().all(1)) and void[0] and torch.equal(a[~void], b[~void])
        if max_ctas:  # (without a budget, how many rows a CTA takes depends on the width)
            assert torch.equal(void, torch.arange(T, device=DEV) % max_ctas == 0)
        else:
            assert int(void.sum()) < T // 8
    again = run(t, inplace, out, max_ctas=max_ctas)
    assert all(a is None or torch.equal(a, b) for a, b in zip(want, again)) and B.moe_comm_error() == 0
