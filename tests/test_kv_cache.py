"""pq_kv_write, pq_kv_read: refusals (CPU) and the cache's contents bit for bit (GPU).

    s = fl32(max |x| fl32(1/448)),  code_i = E(fl32(x_i fl32(1/s))),  read back as fl(code_i s)

The definition rounds each of these binary32 steps, so numpy's binary32 gives the same bits (one division, one product
and one rounding to e4m3 or to the 16-bit type each); there is no tolerance."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
from oracle import e4m3

F16, BF16, U8, F32, I32, I64 = torch.float16, torch.bfloat16, torch.uint8, torch.float32, torch.int32, torch.int64
TYPES = {"f16": F16, "bf16": BF16}
FAKE = 0x100000000   # aligned, never dereferenced: a check fails first or there is nothing to do


def _write(**kw):
    a = dict(k=FAKE, ldk=1024, hsk=128, v=FAKE + (1 << 24), ldv=1024, hsv=128, type=1, T=4, Hkv=8, D=128, slots=FAKE + (2 << 24),
             kc=FAKE + (3 << 24), vc=FAKE + (4 << 24), ks=FAKE + (5 << 24), vs=FAKE + (6 << 24), pages=9, page=16, s=None)
    a.update(kw)
    return pq.lib().pq_kv_write(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(type=2), -2), (dict(type=-1), -2), (dict(D=96), -2), (dict(D=0), -2), (dict(Hkv=0), -2), (dict(Hkv=65537), -2),
    (dict(page=8), -2), (dict(page=24), -2), (dict(page=2048), -2), (dict(page=0), -2), (dict(pages=-1), -2), (dict(pages=2**31), -2),
    (dict(ldk=1028), -2), (dict(hsk=132), -2), (dict(ldv=-8), -2), (dict(hsv=-128), -2), (dict(ldk=2**31), -2),
    (dict(ks=None), -1), (dict(vs=None), -1), (dict(kc=None), -1), (dict(vc=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(slots=None), -1),
    (dict(k=FAKE + 8), -3), (dict(v=FAKE + 2), -3), (dict(kc=FAKE + 8), -3), (dict(vs=FAKE + 2), -3), (dict(slots=FAKE + 4), -3),
    (dict(T=2**31 - 1), -2), (dict(T=0), 0), (dict(T=0, k=None, v=None, slots=None), 0), (dict(pages=0, kc=None, vc=None), 0),
    # an output over an input, or over another output
    (dict(kc=FAKE), -2), (dict(vc=FAKE + (1 << 24) - 16), -2), (dict(kc=FAKE + 2 * (3 * 1024 + 1024) - 16), -2), (dict(vc=FAKE + (3 << 24) + 16), -2),
    (dict(ks=FAKE + (3 << 24) + 64), -2), (dict(vs=FAKE + (5 << 24)), -2), (dict(kc=FAKE + (2 << 24)), -2), (dict(ks=FAKE + (2 << 24) + 16), -2),
])
def test_write_refusals(kw, code):
    assert _write(**kw) == code
    assert bool(pq.lib().pq_last_error()) == (code != 0)


def _read(**kw):
    a = dict(kc=FAKE, vc=FAKE + (1 << 24), ks=FAKE + (2 << 24), vs=FAKE + (3 << 24), pages=9, page=16, table=FAKE + (4 << 24), width=3,
             cu=FAKE + (5 << 24), B=2, T=4, Hkv=8, D=128, k=FAKE + (6 << 24), v=FAKE + (7 << 24), type=0, s=None)
    a.update(kw)
    return pq.lib().pq_kv_read(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), -2), (dict(B=-1), -2), (dict(width=-1), -2), (dict(type=2), -2), (dict(D=32), -2), (dict(Hkv=0), -2), (dict(page=17), -2),
    (dict(pages=-5), -2), (dict(ks=None), -1), (dict(kc=None), -1), (dict(table=None), -1), (dict(cu=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k=FAKE + 8), -3), (dict(cu=FAKE + 2), -3), (dict(table=FAKE + 1), -3), (dict(vc=FAKE + 4), -3), (dict(T=2**31 - 1), -2),
    (dict(T=0), 0), (dict(B=0), 0),
    (dict(k=FAKE + 16), -2), (dict(v=FAKE + (2 << 24)), -2), (dict(v=FAKE + (6 << 24)), -2), (dict(k=FAKE + (4 << 24) + 16), -2), (dict(v=FAKE + (5 << 24)), -2),
    (dict(k=FAKE + (1 << 24) - 2 * 4 * 8 * 128 + 16), -2),
])
def test_read_refusals(kw, code):
    assert _read(**kw) == code
    assert bool(pq.lib().pq_last_error()) == (code != 0)


def _z(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


def _write_args(**kw):
    a = dict(k=_z(4, 8, 128), v=_z(4, 8, 128), slots=_z(4, dtype=I64), k_cache=_z(3, 8, 16, 128, dtype=U8), v_cache=_z(3, 8, 16, 128, dtype=U8),
             k_scale=_z(3, 8, 16, dtype=F32), v_scale=_z(3, 8, 16, dtype=F32))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw,err", [
    (dict(k=None), TypeError), (dict(k=_z(4, 8, 128, dtype=F32)), TypeError), (dict(k=_z(4, 1024)), ValueError), (dict(v=_z(3, 8, 128)), ValueError),
    (dict(v=_z(4, 8, 128, dtype=BF16)), TypeError), (dict(v=_z(4, 8, 64)), ValueError), (dict(k=_z(8, 4, 128).transpose(0, 1).transpose(1, 2)), ValueError),
    (dict(slots=_z(4, dtype=I32)), TypeError), (dict(slots=_z(5, dtype=I64)), ValueError), (dict(k_cache=_z(3, 8, 16, 128)), TypeError),
    (dict(v_cache=_z(2, 8, 16, 128, dtype=U8)), ValueError), (dict(k_cache=_z(3, 4, 16, 128, dtype=U8)), ValueError), (dict(k_cache=_z(3, 16, 128, dtype=U8)), ValueError),
    (dict(k_scale=None), ValueError), (dict(k_scale=_z(3, 8, 16)), TypeError), (dict(v_scale=_z(3, 8, 8, dtype=F32)), ValueError),
    (dict(k_scale=None, v_scale=None), TypeError), (dict(k_scale=None, v_scale=None, k_cache=_z(3, 8, 16, 128), v_cache=_z(3, 8, 16, 128, dtype=BF16)), TypeError),
    (dict(), TypeError),   # the last: CPU tensors
])
def test_write_binding_refusals(kw, err):
    with pytest.raises(err):
        pq.kv_write(**_write_args(**kw))


@pytest.mark.parametrize("kw,err", [
    (dict(block_table=_z(2, 3)), TypeError), (dict(block_table=_z(2, dtype=I32)), ValueError), (dict(cu=_z(2, dtype=I32)), ValueError),
    (dict(cu=_z(3, dtype=I64)), TypeError), (dict(T=-1), ValueError), (dict(T=2**31), ValueError), (dict(dtype=F32), TypeError),
    (dict(out=(_z(4, 8, 128),)), ValueError), (dict(out=(_z(4, 8, 128), _z(4, 8, 128, dtype=BF16))), TypeError),
    (dict(out=(_z(4, 8, 128), _z(4, 8, 128)), dtype=BF16), TypeError), (dict(out=(_z(5, 8, 128), _z(5, 8, 128))), ValueError),
    (dict(k_scale=None, v_scale=None), TypeError), (dict(v_scale=None), ValueError), (dict(k_cache=_z(3, 8, 128, dtype=U8)), ValueError), (dict(), TypeError),
])
def test_read_binding_refusals(kw, err):
    a = dict(k_cache=_z(3, 8, 16, 128, dtype=U8), v_cache=_z(3, 8, 16, 128, dtype=U8), block_table=_z(2, 3, dtype=I32), cu=_z(3, dtype=I32), T=4,
             k_scale=_z(3, 8, 16, dtype=F32), v_scale=_z(3, 8, 16, dtype=F32))
    a.update(kw)
    with pytest.raises(err):
        pq.kv_read(**a)


# ------------------------------------------------------------------------------------------
gpu = pytest.mark.gpu


def _codes(x):
    """Binary32 rows [..., D] -> (codes, scales) by the definition, each step rounded to binary32."""
    x = np.asarray(x, dtype=np.float32)
    finite = np.isfinite(x).all(-1)
    most = np.abs(np.where(finite[..., None], x, 0)).max(-1)
    s = (most * np.float32(1 / 448)).astype(np.float32)
    s = np.where(s < np.finfo(np.float32).tiny, np.float32(0), s)
    with np.errstate(divide="ignore"):
        inv = np.where(s > 0, np.float32(1) / s, np.float32(0)).astype(np.float32)
    codes = e4m3.encode((np.where(finite[..., None], x, 0) * inv[..., None]).astype(np.float32))
    return codes, np.where(finite, s, np.float32(np.nan))


def _same_bits(a, b):
    a, b = np.ascontiguousarray(a), np.ascontiguousarray(b)
    return a.shape == b.shape and np.array_equal(a.view(np.uint8), b.view(np.uint8))


def _rows(g, T, H, D, dtype):
    x = torch.randn((T, H, D), generator=g) * torch.exp(2 * torch.randn((T, H, 1), generator=g))
    x[torch.rand((T, H), generator=g) < 0.05] = 0                                             # empty rows
    return x.to(dtype)


def _place(g, T, pages, page, skip=0.2):
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[torch.rand(T, generator=g) < skip] = -1
    return slots


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("T,Hkv,page,quant", [(1, 1, 16, True), (3, 5, 16, True), (129, 8, 64, True), (517, 3, 256, True), (70, 2, 1024, True),
                                              (1, 8, 16, False), (131, 3, 32, False)])
def test_write(D, kind, T, Hkv, page, quant):
    g, dtype = torch.Generator().manual_seed(T + D), TYPES[kind]
    pages = T // page + 3
    k, v = _rows(g, T, Hkv, D, dtype), _rows(g, T, Hkv, D, dtype)
    slots = _place(g, T, pages, page)
    shape = (pages, Hkv, page, D)
    cache = [torch.randint(0, 120, shape, generator=g, dtype=torch.uint8) if quant else torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
    scale = [torch.rand(shape[:3], generator=g) if quant else None for _ in range(2)]
    dev = [None if c is None else c.cuda() for c in cache + scale]
    got = pq.kv_write(k.cuda(), v.cuda(), slots.cuda(), *dev)
    assert got[0] is dev[0] and got[1] is dev[1]
    for which, x in enumerate((k, v)):
        c, s = cache[which].clone(), None if not quant else scale[which].clone()
        for t in range(T):
            if slots[t] >= 0:
                p, r = int(slots[t]) // page, int(slots[t]) % page
                if quant:
                    codes, sc = _codes(x[t].float().numpy())
                    c[p, :, r], s[p, :, r] = torch.from_numpy(codes), torch.from_numpy(np.ascontiguousarray(sc))
                else:
                    c[p, :, r] = x[t]
        assert torch.equal(dev[which].cpu().view(torch.uint8), c.view(torch.uint8))
        if quant:
            assert _same_bits(dev[2 + which].cpu().numpy(), s.numpy())


@gpu
def test_write_extremes():
    """The ends of the types: largest values, subnormals, negative zeros, values next to an e4m3 border, infinities and NaN."""
    D, inf, nan = 64, float("inf"), float("nan")
    rows = [[3.3895313892515355e38] * D, [2.0 ** -133] * D, [2.0 ** -126, -2.0 ** -130] * (D // 2), [-0.0] * D, [1.0, inf] + [2.0] * (D - 2),
            [nan] + [1.0] * (D - 1), [-inf] * D, [448.0, 17.0, 18.0, 19.0, 232.0, 240.0, -248.0, 2.0 ** -9] * (D // 8),
            [448.0 * 2.0 ** -118] + [2.0 ** -120] * (D - 1)]
    x = torch.tensor(rows, dtype=torch.float32).to(BF16).reshape(len(rows), 1, D)
    kc, vc = (torch.full((1, 1, 16, D), 0xA5, dtype=U8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((1, 1, 16), device="cuda") for _ in range(2))
    pq.kv_write(x.cuda(), (-x).cuda(), torch.arange(len(rows), device="cuda"), kc, vc, ks, vs)
    for c, s, y in ((kc, ks, x), (vc, vs, -x)):
        codes, scales = _codes(y[:, 0].float().numpy())
        assert np.array_equal(c[0, 0, :len(rows)].cpu().numpy(), codes)
        got = s[0, 0, :len(rows)].cpu().numpy()
        assert np.array_equal(got, scales, equal_nan=True) and np.isnan(got[4:7]).all()
        assert bool((c[0, 0, len(rows):] == 0xA5).all())
    table, cu = torch.zeros((1, 1), dtype=I32, device="cuda"), torch.tensor([0, len(rows)], dtype=I32, device="cuda")
    k, _ = pq.kv_read(kc, vc, table, cu, len(rows), ks, vs, dtype=BF16)
    assert torch.isnan(k[4:7]).all() and torch.isfinite(k[[0, 1, 2, 3, 7, 8]]).all()


@gpu
@pytest.mark.parametrize("first", [0, 16])
def test_write_of_a_merged_projections_columns(first):
    """q, k and v as the columns of one buffer, rows apart and heads apart, and slots that are not the cache's."""
    T, Hkv, D, page = 37, 4, 128, 16
    g = torch.Generator().manual_seed(7)
    y = torch.randn((T, first + 3 * 2 * Hkv * D), generator=g).to(BF16).cuda()
    k = y[:, first:first + 2 * Hkv * D].unflatten(1, (Hkv, 2 * D))[:, :, :D]          # every second head-wide column block
    v = y[:, first + 2 * Hkv * D:first + 3 * Hkv * D].unflatten(1, (Hkv, D))
    pages = 4
    slots = torch.randperm(pages * page, generator=g)[:T]
    slots[3], slots[5], slots[8], slots[9] = -1, pages * page, 2 ** 40, -2 ** 63
    a = [torch.zeros((pages, Hkv, page, D), dtype=U8, device="cuda") for _ in range(2)] + [torch.zeros((pages, Hkv, page), device="cuda") for _ in range(2)]
    b = [t.clone() for t in a]
    pq.kv_write(k, v, slots.cuda(), *a)
    live = [t for t in range(T) if 0 <= slots[t] < pages * page]
    pq.kv_write(k[live].contiguous(), v[live].contiguous(), slots[live].cuda(), *b)
    assert len(live) == T - 4 and all(torch.equal(x, y) for x, y in zip(a, b)) and bool(a[0].any())
    with pytest.raises(pq.PQError):      # a row that does not start on a 16-byte line
        pq.kv_write(y[:, 4:4 + Hkv * D].unflatten(1, (Hkv, D)), v, slots.cuda(), *a)
    with pytest.raises(pq.PQError):      # a head stride that does not
        pq.kv_write(y.as_strided((T, Hkv, D), (y.shape[1], D + 4, 1)), v, slots.cuda(), *a)


def _paged_copy(g, lens, Hkv, page, D, kind, spare=3):
    """A cache of sequences on shuffled pages, everything else in it poisoned; (caches, scales, table, rows on the CPU in 64 bits)."""
    need = [-(-n // page) for n in lens]
    pages, width = sum(need) + spare, max(1, max(need, default=1))
    order = torch.randperm(pages, generator=g).to(I32)
    table, at = torch.full((len(lens), width), -1, dtype=I32), 0
    shape = (pages, Hkv, page, D)
    if kind == "e4m3":
        caches = [torch.full(shape, 0x7F, dtype=U8) for _ in range(2)]
        scales = [torch.full(shape[:3], float("nan")) for _ in range(2)]
    else:
        caches, scales = [torch.full(shape, float("nan")).to(TYPES[kind]) for _ in range(2)], [None, None]
    rows = [[], []]
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for w in range(2):
            x = torch.randn((n, Hkv, D), generator=g) * torch.exp(0.5 * torch.randn((n, Hkv, 1), generator=g))
            p, r = table[b].long()[torch.arange(n) // page], torch.arange(n) % page
            if kind == "e4m3":
                codes, s = _codes(x.numpy()) if n else (np.zeros((0, Hkv, D), np.uint8), np.zeros((0, Hkv), np.float32))
                codes, s = torch.from_numpy(codes), torch.from_numpy(np.ascontiguousarray(s))
                caches[w][p, :, r], scales[w][p, :, r] = codes, s
                x = codes.view(torch.float8_e4m3fn).double() * s.double()[..., None]
            else:
                caches[w][p, :, r] = x.to(TYPES[kind])
                x = x.to(TYPES[kind]).double()
            rows[w].append(x)
    return caches, scales, table, rows


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind,out", [("e4m3", "f16"), ("e4m3", "bf16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("lens,Hkv,page", [([1], 1, 16), ([65], 4, 64), ([0, 33, 0, 16, 1, 255, 0], 3, 16), ([300, 1000], 2, 256)])
def test_read(D, kind, out, lens, Hkv, page):
    g = torch.Generator().manual_seed(D + len(lens))
    caches, scales, table, rows = _paged_copy(g, lens, Hkv, page, D, kind)
    ahead, T = 2, sum(lens) + 5                                                # rows of no sequence before and behind
    cu = torch.tensor([ahead + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=I32)
    got = tuple(torch.full((T, Hkv, D), 7.0, dtype=TYPES[out], device="cuda") for _ in range(2))
    dev = [None if s is None else s.cuda() for s in scales]
    res = pq.kv_read(caches[0].cuda(), caches[1].cuda(), table.cuda(), cu.cuda(), T, *dev, out=got)
    assert res is got
    for w in range(2):
        want = torch.cat(rows[w]).float().to(TYPES[out])     # code * s is rounded to binary32, then to the 16-bit type
        y = got[w].cpu()
        assert torch.equal(y[ahead:ahead + sum(lens)].view(torch.int16), want.view(torch.int16))
        assert bool((y[:ahead] == 7).all()) and bool((y[ahead + sum(lens):] == 7).all())
    made = pq.kv_read(caches[0].cuda(), caches[1].cuda(), table.cuda(), cu.cuda(), T, *dev, dtype=TYPES[out])
    assert all(m.dtype == TYPES[out] and torch.equal(m[ahead:T - 3], y[ahead:T - 3]) for m, y in zip(made, got))


@gpu
def test_read_of_pages_that_are_not_the_caches():
    g = torch.Generator().manual_seed(1)
    page, Hkv, D = 16, 2, 64
    caches, scales, table, rows = _paged_copy(g, [80, 40], Hkv, page, D, "e4m3")
    bad = table.clone()
    bad[0, 1], bad[0, 3], bad[1, 0] = -1, caches[0].shape[0], -2 ** 31
    cu = torch.tensor([0, 80, 160], dtype=I32)      # the second passes the table's width in its last rows
    k, v = pq.kv_read(caches[0].cuda(), caches[1].cuda(), bad[:, :3].contiguous().cuda(), cu.cuda(), 160, scales[0].cuda(), scales[1].cuda())
    for y, r in ((k, rows[0]), (v, rows[1])):
        want = torch.zeros(160, Hkv, D, dtype=torch.float64)
        want[:16], want[32:48] = r[0][:16], r[0][32:48]
        want[96:120] = r[1][16:40]
        y = y.cpu()
        assert torch.equal(y[:120], want[:120].float().half()) and bool((y[128:] == 0).all())


@gpu
def test_rows_written_and_read_back_through_pages():
    """Chunks of two sequences written in turn, one of them ending inside a page, read back together."""
    page, Hkv, D, T = 16, 8, 128, 50
    g = torch.Generator().manual_seed(5)
    x = [torch.randn((T, 2, Hkv, D), generator=g).to(BF16).cuda() for _ in range(2)]
    pages = 9
    order = torch.randperm(pages, generator=g)
    table = order[:8].reshape(2, 4).to(I32)
    a = [torch.zeros((pages, Hkv, page, D), dtype=U8, device="cuda") for _ in range(2)] + [torch.zeros((pages, Hkv, page), device="cuda") for _ in range(2)]
    for lo, hi in ((0, 1), (1, 17), (17, 37), (37, 50)):
        for b in range(2):
            at = torch.arange(lo, hi)
            slots = table[b].long()[at // page] * page + at % page
            pq.kv_write(x[b][lo:hi, 0], x[b][lo:hi, 1], slots.cuda(), *a)
    cu = torch.tensor([0, T, 2 * T], dtype=I32, device="cuda")
    k, v = pq.kv_read(a[0], a[1], table.cuda(), cu, 2 * T, a[2], a[3], dtype=BF16)
    for w, y in ((0, k), (1, v)):
        for b in range(2):
            codes, s = _codes(x[b][:, w].float().cpu().numpy())
            want = (torch.from_numpy(codes).view(torch.float8_e4m3fn).float() * torch.from_numpy(np.ascontiguousarray(s))[..., None]).to(BF16)
            assert torch.equal(y[b * T:(b + 1) * T].cpu(), want)
