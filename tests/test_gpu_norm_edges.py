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


@pytest.mark.parametrize("dtype,resid", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                         (torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("H", [256, 1024, 2048, 7168, 16384])
@pytest.mark.parametrize("out", [True, False])
def test_infinities_and_nan(H, dtype, resid, out):
    """By the formulas: a NaN makes its row NaN where it is normed, an infinity makes a norm's other numbers 0 and itself
    NaN; the other rows keep their bits."""
    T = 23
    t = tensors(T, H, dtype, resid, 0)
    want = run(t, out=out, max_ctas=2)
    t["y"][3, H // 2] = float("nan")
    t["y"][7, 0] = float("inf")
    t["resid"][12, H - 1] = float("-inf")
    t["resid"][15, 1] = float("nan")
    t["y"][18] = float("nan")
    ro, o = run(t, out=out, max_ctas=2)
    odd = torch.zeros(T, dtype=torch.bool, device=DEV)
    odd[[3, 7, 12, 15, 18]] = True
    assert torch.equal(ro[~odd], want[0][~odd])
    # the first norm: y's NaN is in every number, y's infinity is NaN beside x = 0, so r' is the residual there
    assert ro[3].isnan().all() and ro[18].isnan().all()
    assert ro[7, 0].isnan() and torch.equal(ro[7, 1:], t["resid"][7, 1:])
    assert ro[12, H - 1] == float("-inf") and torch.equal(ro[12, :H - 1], want[0][12, :H - 1])
    assert ro[15, 1].isnan() and int(ro[15].isnan().sum()) == 1
    if out:
        assert torch.equal(o[~odd], want[1][~odd])
        assert all(o[i].isnan().all() for i in (3, 7, 15, 18))
        assert o[12, H - 1].isnan() and torch.all(o[12, :H - 1] == 0)
    assert B.moe_comm_error() == 0  # numbers, not a wait


def test_infinities_and_nan_in_latent_vectors():
    x = torch.randn(6, 576, device=DEV).to(torch.bfloat16)
    w = torch.randn(512, device=DEV).to(torch.bfloat16)
    slots = torch.arange(6, device=DEV)
    pools = []
    for bad in (False, True):
        if bad:
            x[1, 5], x[3, 0], x[4, 540] = float("nan"), float("inf"), float("nan")
        pool = torch.zeros(1, 16, 576, dtype=torch.bfloat16, device=DEV)
        B.moe_latent_write(B.latent_cache(pool), x[:, :512], x[:, 512:], slots, weight=w)
        pools.append(pool[0])
    good, got = pools
    assert torch.equal(good[[0, 2, 5]], got[[0, 2, 5]]) and torch.equal(good[4, :512], got[4, :512])
    assert got[1, :512].isnan().all() and torch.equal(got[1, 512:], good[1, 512:])
    assert got[3, 0].isnan() and torch.all(got[3, 1:512] == 0)
    assert got[4, 540].isnan() and int(got[4].isnan().sum()) == 1
