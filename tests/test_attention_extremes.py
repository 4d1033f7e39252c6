"""pq_attn_decode and pq_attn_prefill at the ends of what they take: queries that see no key beside values that are not finite, scales that
make one key all of the weight, values at the end of their type, weights far below the largest one. Against the formula in 64 bits.

The tolerances are those of test_attention, but for what each test says."""
import math

import pytest
import torch

import rotated_w4a8_group_amd as pq
import test_attention as ta

pytestmark = pytest.mark.gpu
F16, BF16, U8, I32 = torch.float16, torch.bfloat16, torch.uint8, torch.int32
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


def _i32(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


# ------------------------------------------------------------------------------------------
# (queries, keys): whole items, and items cut along the keys (few items, more than 1024 keys)
NO_KEY = [[(40, 20), (5, 3)], [(300, 200), (9, 9)], [(1300, 1200)], [(150, 100), (1500, 1480), (7, 2000)]]


@pytest.mark.parametrize("lens", NO_KEY)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_without_a_key_beside_values_that_are_not_finite(lens, D, kind, out, bad):
    """Rows that see no key are zeros whatever V holds; those that see keys but no bad value are as without it."""
    g = torch.Generator().manual_seed(D + len(lens))
    q, k, v, cu_q, cu_k = ta._prompts(g, lens, 2, 1, D, ta.TYPES[kind])
    v = v.clone()
    kat, first = 0, []
    for nq, nk in lens:       # a value that the first rows with keys see, one that they do not, and the last
        at = [x for x in (3, 17, 70, nk - 1) if x < nk]
        first.append(min(at))
        for x in at:
            v[kat + x, 0, x % D] = bad
        kat += nk
    o = pq.attn_prefill(q, k, v, cu_q, cu_k, dtype=ta.TYPES[out])
    at = kat = 0
    for (nq, nk), f in zip(lens, first):
        none = max(nq - nk, 0)
        assert bool((o[at:at + none] == 0).all()), (nq, nk)
        sane = max(0, min(nq, f - (nk - nq)))       # rows that see keys 0 .. f - 1 at most
        assert bool(torch.isfinite(o[at:at + sane]).all()) and not bool(torch.isfinite(o[at + sane:at + nq]).all(-1).any()), (nq, nk)
        for h in range(2):
            visible = torch.ones((sane, nk), dtype=torch.bool, device="cuda").tril(nk - nq)
            ref = ta._reference(q[at:at + sane, h].double(), k[kat:kat + nk, 0].double(), torch.nan_to_num(v[kat:kat + nk, 0].double(), 0, 0, 0), D ** -0.5, visible)
            ta._check(o[at:at + sane, h], ref, nk, D, q.dtype, ta._e_p(q, o), f"beside bad values, {(nq, nk)}, head {h}")
        at, kat = at + nq, kat + nk


# ------------------------------------------------------------------------------------------
def _whole_numbers(g, *shape, most=3):
    return torch.randint(-most, most + 1, shape, generator=g).float()


@pytest.mark.parametrize("scale", [1e5, 3e6, 1e8, 1e9, 2.0 ** 40, 2.0 ** 64])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("nq,nk", [(70, 70), (40, 3000)])
def test_prefill_scales_that_leave_one_weight(nq, nk, kind, out, scale):
    """Scores are whole numbers, exactly; those below the largest are at least `scale` below it, where exp gives 0, and equal ones have equal
    weights: the result is the mean over the largest, and scores leave no error."""
    g = torch.Generator().manual_seed(nk)
    D = 64
    k, v = _whole_numbers(g, nk, 1, D).to(ta.TYPES[kind]).cuda(), _whole_numbers(g, nk, 1, D, most=8).to(ta.TYPES[kind]).cuda()
    q = (_whole_numbers(g, nq, 2, D) * 7).to(ta.TYPES[kind]).cuda()
    o = pq.attn_prefill(q, k, v, _i32(0, nq), _i32(0, nk), scale=scale, dtype=ta.TYPES[out])
    visible = torch.ones((nq, nk), dtype=torch.bool, device="cuda").tril(nk - nq)
    for h in range(2):
        a = (q[:, h].double() @ k[:, 0].double().t()).masked_fill(~visible, -math.inf)
        top = (a == a.amax(-1, keepdim=True)).double()
        want, A = (top @ x / top.sum(-1, keepdim=True) for x in (v[:, 0].double(), v[:, 0].double().abs()))
        tol = ta.E[o.dtype] * want.abs() + 1.01 * ta._e_p(q, o) * (A + want.abs()) + (4 * nk + 8) * U * A + 2.0 ** -25
        err = (o[:, h].double() - want).abs()
        assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the tolerance"


def _cache(g, n, D, kind, k, v, page=16):
    """k, v [n, 1, D] on pages of their own: values that e4m3 holds, under scales that are powers of two."""
    pages = -(-n // page)
    order = torch.randperm(pages, generator=g)
    at = torch.arange(n)
    out, scales = [], []
    for x, s in ((k, 0.5), (v, 2.0)):
        c = torch.full((pages, 1, page, D), math.nan).to(E4M3 if kind == "e4m3" else ta.TYPES[kind])
        y = (x / s).to(c.dtype) if kind == "e4m3" else x.to(c.dtype)
        c.view(U8 if kind == "e4m3" else torch.int16)[order[at // page], :, at % page] = y.view(U8 if kind == "e4m3" else torch.int16)
        out.append((c.view(U8) if kind == "e4m3" else c).cuda())
        scales.append(torch.full((pages, 1, page), s, device="cuda") if kind == "e4m3" else None)
    return out, order.to(I32)[None].cuda(), scales


@pytest.mark.parametrize("scale", [1e5, 1e8, 1e9, 2.0 ** 40, 2.0 ** 64])
@pytest.mark.parametrize("cache,kind", [("e4m3", "bf16"), ("e4m3", "f16"), ("f16", "f16"), ("bf16", "bf16")])
@pytest.mark.parametrize("n", [37, 700, 9001])
def test_decode_scales_that_leave_one_weight(n, cache, kind, scale):
    """The same for single tokens, whose weights are held in two pieces."""
    g = torch.Generator().manual_seed(n)
    D, Hq = 64, 20
    k, v = _whole_numbers(g, n, 1, D), _whole_numbers(g, n, 1, D, most=8)
    q = (_whole_numbers(g, 1, Hq, D) * 7).to(ta.TYPES[kind]).cuda()
    c, table, s = _cache(g, n, D, cache, k, v)
    o = pq.attn_decode(q, *c, table, _i32(n), *s, scale=scale)
    a = q[0].double() @ k[:, 0].double().cuda().t()
    top = (a == a.amax(-1, keepdim=True)).double()
    want = top @ v[:, 0].double().cuda() / top.sum(-1, keepdim=True)
    A = top @ v[:, 0].double().abs().cuda() / top.sum(-1, keepdim=True)
    tol = ta.E[o.dtype] * want.abs() + 1.01 * 2.0 ** -16 * (A + want.abs()) + (4 * n + 8) * U * A + 2.0 ** -25
    err = (o[0].double() - want).abs()
    assert bool((err <= tol).all()), f"{float((err / tol).max()):.3g} of the tolerance"


# ------------------------------------------------------------------------------------------
def _ends(g, n, D):
    """Values up to the largest that bf16 holds, both signs, and ordinary ones."""
    x = (2 * torch.rand((n, 1, D), generator=g) - 1) * 3.38e38
    x[:, :, 1] = 3.3895313892515355e38
    x[:, :, 2::4] = torch.randn((n, 1, len(range(2, D, 4))), generator=g)
    x[:, :, 3::4] *= 1e-20
    return x


@pytest.mark.parametrize("scale", [1e-6, 0.125, 3.0])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens", [[300, 40, 1], [700, 20], [5000, 300]])
def test_decode_largest_values(lens, D, cache, scale):
    """A mean of finite values is finite, whatever their sum is: equal weights, and a maximum that keeps rising along the keys."""
    g = torch.Generator().manual_seed(sum(lens) + D)
    page = 16
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g).to(I32)
    table = torch.full((len(lens), max(need)), -1, dtype=I32)
    kc = torch.full((pages, 1, page, D), math.nan, dtype=BF16)
    vc, vs = kc.clone(), torch.full((pages, 1, page), math.nan)
    ks, code = vs.clone(), [torch.full((pages, 1, page, D), 0x7F, dtype=U8) for _ in range(2)]
    rows, at = [[], []], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        k = torch.randn((n, 1, D), generator=g)
        k[:, 0, 0] = torch.linspace(-40, 40, n)
        v = _ends(g, n, D) if b < 2 else torch.randn((n, 1, D), generator=g)
        p, r = table[b].long()[torch.arange(n) // page], torch.arange(n) % page
        for w, x in enumerate((k, v)):
            if cache == "e4m3":
                s = x.abs().amax(-1) / 448
                c = (x / s[..., None]).to(E4M3)
                code[w][p, :, r], (ks, vs)[w][p, :, r] = c.view(U8), s
                rows[w].append(c.double() * s.double()[..., None])
            else:
                x = x.to(BF16)
                (kc, vc)[w][p, :, r] = x
                rows[w].append(x.double())
    q = torch.randn((len(lens), 4, D), generator=g)
    q[:, :, 0] = 30
    q = q.to(BF16).cuda()
    dev = [c.cuda() for c in (code if cache == "e4m3" else (kc, vc))]
    sc = [ks.cuda(), vs.cuda()] if cache == "e4m3" else [None, None]
    o = pq.attn_decode(q, *dev, table.cuda(), _i32(*lens), *sc, scale=scale)
    assert bool(torch.isfinite(o).all())
    ta._check_decode(o, q, rows, lens, float(torch.tensor(scale, dtype=torch.float32)), "largest values")


@pytest.mark.parametrize("scale", [1e-6, 0.125, 3.0])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("nq,nk", [(70, 70), (20, 3000)])
def test_prefill_largest_values(nq, nk, D, scale):
    g = torch.Generator().manual_seed(nk + D)
    k = torch.randn((nk, 1, D), generator=g)
    k[:, 0, 0] = torch.linspace(-40, 40, nk)
    q = torch.randn((nq, 2, D), generator=g)
    q[:, :, 0] = 30
    q, k, v = q.to(BF16).cuda(), k.to(BF16).cuda(), _ends(g, nk, D).to(BF16).cuda()
    o = pq.attn_prefill(q, k, v, _i32(0, nq), _i32(0, nk), scale=scale)
    assert bool(torch.isfinite(o).all())
    ta._check_prompts(o, q, k, v, [(nq, nk)], 0, True, float(torch.tensor(scale, dtype=torch.float32)), "largest values")


# ------------------------------------------------------------------------------------------
LN2 = float(torch.tensor(math.log(2), dtype=torch.float32))   # as a scale: its product with log2(e) rounds to 1 in binary32
GAPS = [0.0, 8.0, 14.5, 17.5, 20.5, 23.5, 25.0, 27.0]          # powers of two between one key's weight and every other's


def _one_large(g, n, D, at):
    """q [1, heads, D], k, v [n, 1, D]: with scale LN2 head h's weights are 1 at the keys `at` and 2^-GAPS[h] at all others; the first kind's values are 0,
    the others' have a mean of about 1.5: the output is what the small weights sum to."""
    k, v = torch.zeros((n, 1, D)), torch.randint(0, 4, (n, 1, D), generator=g).float()
    k[at, 0, 0], v[at] = 1, 0
    q = torch.zeros((1, len(GAPS), D))
    q[0, :, 0] = torch.tensor(GAPS)
    return q.to(F16).cuda(), k, v


def _check_small_weights(o, q, k, v, e_p, floor, what):
    """test_attention's tolerance but for two terms. `floor`: what rounding takes from a weight at most, relative to the largest (there 2^-25).
    (4 n + 8) u is for sums of n terms in any order; here n is 1e5, and no chain of additions is longer than a lane's keys, a quarter of its wave's,
    which has half of them at most, and one for each wave and piece: (n / 8 + 1200) u between both sums."""
    n, D = k.shape
    want, Q, A, S = ta._reference(q.double(), k.double(), v.double(), LN2, torch.ones((q.shape[0], n), dtype=torch.bool, device="cuda"))
    tol = ta.E[o.dtype] * want.abs() + 1.01 * (2 * (2 * (2 * D + 4) * U * Q + 4 * U) + (n / 8 + 1200) * U) * A + 1.01 * e_p * (A + want.abs()) + 2.0 ** -25
    tol = tol + 1.01 * floor * (S + n * want.abs())
    worst = ((o.double() - want).abs() / tol).amax(-1)
    assert bool((worst <= 1).all()), f"{what}: {[f'{float(w):.2f}' for w in worst]} of the tolerance"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("at", [0, 70000, 131070])
@pytest.mark.parametrize("beside", [0, 520])
def test_prefill_weights_far_below_the_largest(D, at, beside):
    """f16 weights, taken 2^7 times as large, so that 2^-25 is 2^-32 of the largest: cut along the keys, and whole beside many other sequences."""
    g, n = torch.Generator().manual_seed(D), 131071
    q, k, v = _one_large(g, n, D, at)
    more = torch.ones((beside, 1, D))
    o = pq.attn_prefill(torch.cat([q] + [q] * beside), torch.cat([k, more]).to(F16).cuda(), torch.cat([v, more]).to(F16).cuda(),
                        torch.arange(beside + 2, dtype=I32, device="cuda"), _i32(0, *range(n, n + beside + 1)), scale=LN2)
    _check_small_weights(o[0], q[0], k[:, 0].cuda(), v[:, 0].cuda(), 2.0 ** -11, 2.0 ** -32, "prefill")
    assert bool((o[1:] == 1).all())


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("at", [(0,), (0, 32768, 65536, 98304), (131070,)])
@pytest.mark.parametrize("B", [1, 2048])
def test_decode_weights_far_below_the_largest(D, at, B):
    """An f16 cache: both pieces of a weight are f16, taken 2^7 times as large as the weight, so 2^-25 is 2^-32 of the largest. One sequence,
    cut into pieces that most hold small weights only, and so many on the same pages that each is whole, with a large one in each wave's part."""
    g, n = torch.Generator().manual_seed(D), 131071
    q, k, v = _one_large(g, n, D, list(at))
    c, table, _ = _cache(g, n, D, "f16", k, v)
    o = pq.attn_decode(q.expand(B, -1, -1).contiguous(), *c, table.expand(B, -1).contiguous(), torch.full((B,), n, dtype=I32, device="cuda"), scale=LN2)
    _check_small_weights(o[0], q[0], k[:, 0].cuda(), v[:, 0].cuda(), 2.0 ** -16, 2.0 ** -32, "decode")
    assert torch.equal(o, o[:1].expand(B, -1, -1))


def test_head_size_zero_is_refused_on_a_stream_too():
    z, s = torch.zeros((2, 4, 0), dtype=F16, device="cuda"), torch.cuda.current_stream()
    c, t = torch.zeros((3, 4, 16, 0), dtype=F16, device="cuda"), torch.zeros((2, 1), dtype=I32, device="cuda")
    for stream in (None, s):
        with pytest.raises(pq.PQError):
            pq.attn_decode(z, c, c.clone(), t, _i32(1, 1), stream=stream)
        with pytest.raises(pq.PQError):
            pq.attn_prefill(z, z, z.clone(), _i32(0, 2), stream=stream)


# ------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("nq,nk", [(50, 50), (40, 3000)])
def test_prefill_infinite_values_keep_their_sign(kind, D, bad, nq, nk):
    """An infinite value that a row sees, at scores whose weights are far from binary32's ends: that infinity in its channel, whole and cut."""
    g = torch.Generator().manual_seed(D)
    q, k, v, cu_q, cu_k = ta._prompts(g, [(nq, nk)], 4, 2, D, ta.TYPES[kind])
    at = nk - 15                                             # seen from row nq - 15 on, by the heads of key head 0
    v[at, 0, 5] = bad
    o = pq.attn_prefill(q, k, v, cu_q, cu_k, scale=0.02)
    rest = [c for c in range(D) if c != 5]
    seen = o[nq - 15:, :2]
    assert bool(torch.isnan(seen[:, :, 5]).all()) if math.isnan(bad) else bool((seen[:, :, 5] == bad).all())
    assert bool(torch.isfinite(seen[:, :, rest]).all()) and bool(torch.isfinite(o[:nq - 15]).all()) and bool(torch.isfinite(o[:, 2:]).all())


@pytest.mark.parametrize("nq,nk", [(50, 50), (40, 3000)])
def test_prefill_infinite_values_of_no_weight(nq, nk):
    """An infinite value whose weight is below what binary32 holds: NaN in its channel, as 0 times an infinity is, and nothing in others."""
    g = torch.Generator().manual_seed(3)
    q, k, v, cu_q, cu_k = ta._prompts(g, [(nq, nk)], 2, 1, 64, BF16)
    k[:, 0], q[:, :, 0], v[0, 0, 5] = 0, 8, math.inf
    k[1:, 0, 0] = 8                                          # key 0 is 64 scale below all others
    o = pq.attn_prefill(q, k, v, cu_q, cu_k, scale=4.0)
    seen = o[1 if nq == nk else 0:]                          # row 0 of the first sees key 0 alone
    assert bool(torch.isnan(seen[:, :, 5]).all()) and bool(torch.isfinite(o[:, :, :5]).all()) and bool(torch.isfinite(o[:, :, 6:]).all())
    if nq == nk:
        assert bool((o[0, :, 5] == math.inf).all())


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [300, 5000])
def test_decode_a_large_value_of_every_weight(n, D, cache):
    """One key's values of 1e35 under weights of 1 down to 2^-120 of the others', which have ordinary ones, in heads of one product: those whose sums
    are large leave the others' small weights as they are."""
    g = torch.Generator().manual_seed(n)
    gaps = [0.0, 20.0, 40.0, 60.0, 70.0, 80.0, 90.0, 100.0, 110.0, 120.0]
    k, v = torch.zeros((n, 1, D)), torch.randint(-4, 5, (n, 1, D), generator=g).float()
    k[n // 3, 0, 0], v[n // 3] = -1, torch.where(torch.rand((1, D), generator=g) < 0.5, 1.0, 0.5) * 2.0 ** 116
    q = torch.zeros((1, len(gaps), D))
    q[0, :, 0] = torch.tensor(gaps)
    c, table, s = _cache(g, n, D, "bf16", k, v)
    if cache == "e4m3":
        c, table, s = _cache(g, n, D, cache, k, torch.where(v.abs() > 4, v * 2.0 ** -116, v))
        at = (n // 3) // 16
        s[1][table[0, at], 0, n // 3 % 16] *= 2.0 ** 116
    o = pq.attn_decode(q.to(BF16).cuda(), *c, table, _i32(n), *s, scale=LN2)
    ta._check_decode(o, q.to(BF16).cuda(), [[k.double()], [v.double()]], [n], LN2, "a large value")
