"""The paged cache on the GPU: written and read back, bit for bit against a plain
implementation, for types, head layouts, page sizes, strides, padding and bad slots."""
import numpy as np
import pytest
import torch

from moe_expert_dispatch_route_gb300 import binding as B
from serve_ref import E4M3, dequantise, quantise

pytestmark = pytest.mark.gpu
DEV = "cuda"


def pools(pages, H, page, D, dtype, order="hnd"):
    shape = (pages, H, page, D) if order == "hnd" else (pages, page, H, D)
    t = [torch.full(shape, 1.5, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    sc = [None, None]
    if dtype == "e4m3":
        t = [x.to(E4M3) for x in t]
        sc = [torch.full((pages, H, page), 130, dtype=torch.uint8, device=DEV) for _ in range(2)]
    if order != "hnd":
        t = [x.transpose(1, 2) for x in t]
    return t, sc, B.kv_cache(t[0], t[1], sc[0], sc[1])


def raw(t):
    return (t.view(torch.uint8) if t.dtype == E4M3 else t.contiguous().view(torch.int16)).cpu().numpy()


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,H,page,order", [(1, 1, 16, "hnd"), (7, 3, 32, "nhd"), (333, 8, 64, "hnd"),
                                            (1000, 2, 256, "nhd"), (5000, 8, 16, "hnd")])
def test_write(dtype, D, T, H, page, order):
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 3
    (k, v), sc, cache = pools(pages, H, page, D, dtype, order)
    before = [raw(k).copy(), raw(v).copy()]
    x = rng.standard_normal((T, 3 * H, D)) * np.exp(rng.uniform(-12, 12, size=(T, 3 * H, 1)))
    x[0, H] = 0.0
    qkv = torch.tensor(x).to(torch.bfloat16).to(DEV)
    slots = rng.permutation(pages * page)[:T]
    slots[T // 3] = -1 if T > 3 else slots[T // 3]  # padding
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_kv_write(cache, qkv[:, H:2 * H], qkv[:, 2 * H:], torch.tensor(slots, device=DEV), err_flag=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    for i, pool in enumerate((k, v)):
        want, part = before[i], qkv[:, (i + 1) * H:(i + 2) * H]
        if dtype == "bf16":
            val = part.contiguous().view(torch.int16).cpu().numpy()
        else:
            val, s = quantise(part.double().cpu().numpy())
            ws = np.full((pages, H, page), 130, dtype=np.uint8)
        for t in range(T):
            if slots[t] >= 0:
                want[slots[t] // page, :, slots[t] % page] = val[t]
                if dtype == "e4m3":
                    ws[slots[t] // page, :, slots[t] % page] = s[t]
        assert np.array_equal(raw(pool), want)
        if dtype == "e4m3":
            assert np.array_equal(sc[i].cpu().numpy(), ws)


def test_write_extreme_values():
    """The scale's limits, subnormals, infinities and NaN."""
    rows = torch.zeros(8, 1, 64, dtype=torch.bfloat16)
    rows[0, 0, :3] = torch.tensor([3.3895e38, -1e38, 1.0])       # above 448 * 2^119: saturates
    rows[1, 0, :3] = torch.tensor([9.2e-41, 0.0, -9.2e-41])      # subnormal, below the smallest scale
    rows[2, 0, :3] = torch.tensor([2.0**-100 * 448, 2.0**-105, -2.0**-109])
    rows[3, 0, :2] = torch.tensor([448.0, 1.0])
    rows[4, 0, :2] = torch.tensor([450.0, 1.0])                  # rounds to 450 in bf16: the next scale
    rows[5, 0, :2] = torch.tensor([float("inf"), -float("inf")])
    rows[6, 0, 5] = float("nan")
    (k, v), sc, cache = pools(1, 1, 16, 64, "e4m3")
    x = rows.to(DEV)
    B.moe_kv_write(cache, x, x, torch.arange(8, device=DEV))
    codes, s = k.view(torch.uint8)[0, 0].cpu().numpy(), sc[0][0, 0].cpu().numpy()
    want, ws = quantise(rows[:5, 0].double().numpy())
    assert np.array_equal(codes[:5], want) and np.array_equal(s[:5], ws)
    assert ws[0] == 246 and ws[1] == 27 and ws[3] == 127 and ws[4] == 128
    assert codes[5, 0] == 0x7E and codes[5, 1] == 0xFE and s[5] == 246
    assert s[6] == 255 and s[7] == 127 and (codes[7] == 0).all()
    out = [torch.empty(8, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)
    B.moe_kv_read(cache, i32([[0]]), i32([0]), i32([0, 8]), out[0], out[1])
    got = out[0].double().cpu().numpy()[:, 0]
    assert np.array_equal(got[:6], dequantise(codes[:6], s[:6])) and np.isnan(got[6]).all() and (got[7] == 0).all()


def test_write_bad_slot_and_empty():
    (k, v), _, cache = pools(2, 2, 16, 64, "bf16")
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_kv_write(cache, x[:0], x[:0], torch.empty(0, dtype=torch.int64, device=DEV), err_flag=err)
    B.moe_kv_write(cache, x, x, torch.tensor([4, 32, 1 << 40], device=DEV), err_flag=err)
    assert int(err.item()) == 7
    assert int((k != 1.5).any(-1).sum()) == 2 and torch.all(k[0, :, 4] == 1)  # the good slot's two heads


def test_offsets_past_32_bits():
    """A pool of more than 2^31 elements: its last page is written, read back and attended over."""
    pages, page, H, D = 70000, 64, 4, 128
    k = torch.zeros(pages, H, page, D, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    assert k.numel() > 1 << 31
    cache = B.kv_cache(k, v)
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn(2, page, H, D, generator=g, device=DEV).to(torch.bfloat16)
    at = (pages - 1) * page + torch.arange(page, device=DEV)
    B.moe_kv_write(cache, x[0], x[1], at)
    assert torch.equal(k[-1], x[0].transpose(0, 1)) and torch.equal(v[-1], x[1].transpose(0, 1))
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    out = torch.empty_like(x)
    B.moe_kv_read(cache, i32([[pages - 1]]), i32([0]), i32([0, page]), out[0], out[1])
    assert torch.equal(out, x)
    q = torch.zeros(1, H, D, dtype=torch.bfloat16, device=DEV)
    o = torch.empty_like(q)
    ws = torch.zeros(B.moe_attn_workspace_size(cache, H), dtype=torch.uint8, device=DEV)
    B.moe_attn_paged(cache, B.attn_args(q, o, i32([0, 1]), i32([page]), i32([[pages - 1]]), 1, page, 1.0,
                                        workspace=ws))
    mean = x[1].double().mean(0)  # equal scores: p = 1/64 is exact, o is rounded once
    assert torch.all((o[0].double() - mean).abs() <= 2.0**-8 * mean.abs() + 1e-6)


def test_writes_of_more_than_32_bits_of_threads():
    """2^27 + 8 tokens of one head, all but a few of them padding: the last ones are written."""
    T = (1 << 27) + 8
    (k, v), _, cache = pools(1, 1, 16, 128, "bf16")
    x = torch.arange(2, dtype=torch.bfloat16, device=DEV)[:, None, None].expand(2, 1, 128).contiguous()
    slots = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slots[-5:] = torch.arange(5, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    # every token the same row: token stride 0
    B.moe_kv_write(cache, x[0].expand(T, 1, 128), x[1].expand(T, 1, 128), slots, err_flag=err)
    assert int(err.item()) == 0
    assert torch.all(k[0, 0, :5] == 0) and torch.all(v[0, 0, :5] == 1) and torch.all(k[0, 0, 5:] == 1.5)


def test_reads_of_more_than_32_bits_of_threads():
    """2^29 + 40 rows of one head, the same cached tokens over and over: the last ones are written."""
    if torch.cuda.mem_get_info()[0] < 180 << 30:
        pytest.skip("needs 137 GB")
    T, page = (1 << 29) + 40, 64
    k = torch.randn(1, 1, page, 64, device=DEV).to(torch.bfloat16)
    v = torch.randn(1, 1, page, 64, device=DEV).to(torch.bfloat16)
    out = [torch.empty(T, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for o in out:
        o[-100:] = 9.0
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    table = torch.zeros(1, T // page + 1, dtype=torch.int32, device=DEV)
    B.moe_kv_read(B.kv_cache(k, v), table, i32([0]), i32([0, T - 3]), out[0], out[1], err_flag=err)
    assert int(err.item()) == 0
    at = torch.arange(T - 100, T - 3, device=DEV) % page
    for o, pool in ((out[0], k), (out[1], v)):
        assert torch.equal(o[-100:-3, 0], pool[0, 0, at]) and torch.all(o[-3:] == 9.0)


@pytest.mark.parametrize("dtype", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("H,page,order", [(1, 16, "hnd"), (3, 32, "nhd"), (8, 128, "hnd")])
def test_read(dtype, D, H, page, order):
    rng = np.random.default_rng(H)
    lens, start = [5, 0, 1, 300, 64, 0, 33], [0, 3, 17, 250, 64, 1, 31]
    need = [-(-(a + n) // page) for a, n in zip(start, lens)]
    pages = sum(need) + 1
    (k, v), sc, cache = pools(pages, H, page, D, dtype, order)
    for i, t in enumerate((k, v)):
        val = torch.tensor(rng.standard_normal((pages, H, page, D)) * 50, device=DEV)
        if dtype == "bf16":
            t.copy_(val)
        else:
            t.view(torch.uint8).copy_(val.clamp(-448, 448).to(E4M3).view(torch.uint8))
            sc[i].copy_(torch.tensor(rng.integers(27, 247, size=(pages, H, page)), device=DEV))
    perm = rng.permutation(pages)
    table = np.full((len(lens), max(need)), -1, dtype=np.int32)
    at = 0
    for b, m in enumerate(need):
        table[b, :m] = perm[at:at + m]
        at += m
    T = sum(lens)
    cu = np.cumsum([0] + lens)
    i32 = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)
    out = [torch.full((T + 2, H, D), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    B.moe_kv_read(cache, i32(table), i32(start), i32(cu), out[0], out[1], err_flag=err)
    assert int(err.item()) == 0
    for i, t in enumerate((k, v)):
        if dtype == "bf16":
            val = t.double().cpu().numpy()
        else:
            val = dequantise(t.view(torch.uint8).cpu().numpy(), sc[i].cpu().numpy())
        want = np.full((T + 2, H, D), 9.0)
        for b, (a, n) in enumerate(zip(start, lens)):
            for j in range(n):
                want[cu[b] + j] = val[table[b, (a + j) // page], :, (a + j) % page]
        assert np.array_equal(out[i].double().cpu().numpy(), want)


def test_read_bad_pages():
    (k, v), _, cache = pools(4, 1, 16, 64, "bf16")
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)
    out = [torch.full((40, 1, 64), 9.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    # page 99 is outside the pool, tokens 32.. are past the table, start -2 is before the first
    B.moe_kv_read(cache, i32([[1, 99], [2, 3], [0, 1]]), i32([12, 28, -2]), i32([0, 8, 16, 20]), *out, err_flag=err)
    assert int(err.item()) == 7
    got = (out[0][:, 0, 0] == 1.5).cpu().numpy()
    assert got[:4].all() and not got[4:8].any() and got[8:12].all() and not got[12:18].any() and got[18:20].all()
    assert not got[20:].any() and torch.equal(out[0], out[1])
