"""Kernels that a call of moe_attn_latent launches: the second one joins the parts of split tiles, and is left out where
there can be none."""
import ctypes

import pytest
import torch

from latent_ref import attention, chain, check
from moe_expert_dispatch_route_gb300 import binding as B

pytestmark = pytest.mark.gpu
DEV = "cuda"


def kernels(call):
    """Nodes of the graph that the call, captured, leaves."""
    cuda, stream = ctypes.CDLL("libcuda.so.1"), torch.cuda.Stream()
    at, graph, nodes = ctypes.c_void_p(stream.cuda_stream), ctypes.c_void_p(), ctypes.c_size_t()
    torch.cuda.synchronize()
    assert cuda.cuStreamBeginCapture_v2(at, 2) == 0  # CU_STREAM_CAPTURE_MODE_RELAXED
    try:
        call(stream)
    finally:
        status = cuda.cuStreamEndCapture(at, ctypes.byref(graph))
    assert status == 0 and cuda.cuGraphGetNodes(graph, None, ctypes.byref(nodes)) == 0
    cuda.cuGraphDestroy(graph)
    return nodes.value


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("max_kv,max_ctas,want", [(1, 0, 1), (128, 0, 1), (129, 0, 1), (256, 0, 1), (257, 0, 2), (5000, 0, 2),
                                                  (5000, 1, 1), (5000, 4, 2)])
def test_kernels_of_a_call(heads, max_kv, max_ctas, want):
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    pages = -(-max_kv // 64)
    pool = torch.randn(pages, 64, 576, device=DEV).to(torch.bfloat16)
    cache = B.latent_cache(pool)
    q = torch.randn(3, heads, 576, device=DEV).to(torch.bfloat16)
    o = torch.empty(3, heads, 512, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, heads, device=DEV)
    ws = torch.zeros(B.moe_attn_latent_workspace_size(cache, heads), dtype=torch.uint8, device=DEV)
    table = torch.arange(pages, dtype=torch.int32, device=DEV).expand(3, pages).contiguous()
    args = B.attn_latent_args(q, o, i32([0, 1, 2, 3]), i32([max_kv, 1, max_kv // 2]), table, 1, max_kv, 0.07, lse=lse,
                              workspace=ws)
    run = lambda s=None: B.moe_attn_latent(cache, args, max_ctas=max_ctas, stream=s)
    run()
    torch.cuda.synchronize()
    got = o.clone()
    assert kernels(run) == want
    for b, n in enumerate((max_kv, 1, max_kv // 2)):  # what is split and what is not is whole
        kv = pool.view(-1, 576)[:n].double().cpu().numpy()
        ref = attention(q[b:b + 1].double().cpu().numpy(), kv, kv[:, :512], chain(1, n), 0.07)
        check(got[b:b + 1].double().cpu().numpy(), lse[b:b + 1].double().cpu().numpy(), ref, f"{n} keys")
