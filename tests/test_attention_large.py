"""The cache and attention where element and byte offsets pass 32 bits, against the tests' own formulas (GPU, up to about 40 GB of
device memory; only the pages in use are written)."""
import pytest
import torch

import rotated_w4a8_group_amd as pq
import test_attention as ta
import test_kv_cache as tk

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ["e4m3", "bf16"])
def test_cache_past_4_gib(kind):
    """4.5e9 values in each of K and V; the sequence lies on the last pages, the first and those around 2^31 and 2^32 values."""
    page, Hkv, D, pages = 64, 8, 256, 34500
    per = Hkv * page * D
    assert pages * per > 2 ** 32 + 2 ** 27
    used = [pages - 1, 0, pages - 2, 2 ** 31 // per, 2 ** 31 // per - 1, 2 ** 32 // per, 2 ** 32 // per + 1, 5]
    n, Hq = len(used) * page - 3, 16
    g = torch.Generator().manual_seed(1)
    x = [torch.randn((n, Hkv, D), generator=g).bfloat16().cuda() for _ in range(2)]
    dtype = torch.uint8 if kind == "e4m3" else torch.bfloat16
    cache = [torch.empty((pages, Hkv, page, D), dtype=dtype, device="cuda") for _ in range(2)]
    scales = [torch.empty((pages, Hkv, page), device="cuda") for _ in range(2)] if kind == "e4m3" else [None, None]
    table = torch.tensor([used], dtype=I32, device="cuda")
    at = torch.arange(n, device="cuda")
    pq.kv_write(x[0], x[1], table[0].long()[at // page] * page + at % page, *cache, *scales)
    k, v = pq.kv_read(*cache, table, ta._cu([n]), n, *scales, dtype=torch.bfloat16)
    rows = [[], []]
    for w, got in ((0, k), (1, v)):
        if kind == "e4m3":
            codes, s = tk._codes(x[w].float().cpu().numpy())
            want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double() * torch.from_numpy(s.copy()).double()[..., None]
            assert torch.equal(got.cpu(), want.float().bfloat16())
        else:
            want = x[w].double()
            assert torch.equal(got, x[w])
        rows[w].append(want)
    q = ta._heads(g, 1, Hq, D, torch.bfloat16)
    o = pq.attn_decode(q, *cache, table, torch.tensor([n], dtype=I32, device="cuda"), *scales, dtype=torch.float16)
    ta._check_decode(o, q, rows, [n], D ** -0.5, "past 4 GiB")


def test_rows_past_2_31_elements():
    """Prompts whose q, k and v are columns of a buffer of 4.4e9 elements, the last sequence past 2^32 of them."""
    T, ld, D, Hq, Hkv = 66000, 65536, 128, 4, 2
    y = torch.empty((T, ld), dtype=torch.bfloat16, device="cuda")
    assert y.numel() > 2 ** 32
    q, k, v = (y[:, c * D:(c + h) * D].unflatten(1, (h, D)) for c, h in ((0, Hq), (200, Hkv), (510, Hkv)))
    g = torch.Generator().manual_seed(2)
    tail = 300
    for t, h in ((q, Hq), (k, Hkv), (v, Hkv)):
        t.zero_()
        t[T - tail:] = ta._heads(g, tail, h, D, torch.bfloat16)
    lens = [T - tail - 1000, 1000, 170, 130]
    o = torch.full((T, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, T - tail - 1000, T - tail, T - 130, T], dtype=I32, device="cuda")[1:].contiguous()   # the long empty-looking one is left out
    pq.attn_prefill(q, k, v, cu, out=o)
    ta._check_prompts(o[T - tail:], q[T - tail:], k[T - tail:], v[T - tail:], [(170, 170), (130, 130)], 0, True, D ** -0.5, "past 2^32")
    assert not bool(o[T - tail - 1000:T - tail].any()) and bool((o[:T - tail - 1000] == 7).all()) and lens[1] == 1000
    # the same rows into a cache
    cache = [torch.zeros((20, Hkv, 16, D), dtype=torch.uint8, device="cuda") for _ in range(2)] + [torch.zeros((20, Hkv, 16), device="cuda") for _ in range(2)]
    slots = torch.full((T,), -1, dtype=torch.int64, device="cuda")
    slots[T - tail:] = torch.arange(tail, device="cuda")
    pq.kv_write(k, v, slots, *cache)
    kr, vr = pq.kv_read(*cache[:2], torch.arange(20, dtype=I32, device="cuda")[None], ta._cu([tail]), tail, *cache[2:], dtype=torch.bfloat16)
    for got, rows in ((kr, k), (vr, v)):
        codes, s = tk._codes(rows[T - tail:].float().cpu().numpy())
        assert torch.equal(got.cpu(), (torch.from_numpy(codes).view(torch.float8_e4m3fn).float() * torch.from_numpy(s.copy())[..., None]).bfloat16())


def test_the_widest_table():
    """2^31 - 16 positions that a table could hold, a thousand that the sequence has."""
    width, n, D = 2 ** 27 - 1, 1000, 64
    g = torch.Generator().manual_seed(3)
    x = [torch.randn((n, 1, D), generator=g).bfloat16().cuda() for _ in range(2)]
    cache = [torch.empty((64, 1, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    pq.kv_write(*x, torch.arange(n, device="cuda"), *cache)
    table = torch.full((1, width), -1, dtype=I32, device="cuda")
    table[0, :64] = torch.arange(64, dtype=I32, device="cuda")
    q = ta._heads(g, 1, 4, D, torch.bfloat16)
    o = pq.attn_decode(q, *cache, table, torch.tensor([n], dtype=I32, device="cuda"))
    ta._check_decode(o, q, [[t.double()] for t in x], [n], D ** -0.5, "widest table")
    k, v = pq.kv_read(*cache, table, ta._cu([n]), n)
    assert torch.equal(k, x[0]) and torch.equal(v, x[1])
