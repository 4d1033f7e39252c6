"""pq_attn_decode, pq_attn_prefill: refusals (CPU) and parity with the formula in 64 bits (GPU).

    o[h] = sum_j p_j v_j,  p = softmax_j(scale q[h] . k_j) over the keys that the query sees

Tolerance, with u = 2^-24, c = scale, n keys, and in 64 bits Q = max_j c sum_i |q_i k_ji|, A = sum_j p_j |v_j|, e(t) = eps / 2 of a type
(half a step: bf16 2^-8, f16 2^-11).
 - A score is a sum of D exact products in binary32, in any order, by an adder that may truncate: 2 (D - 1) u of the sum of magnitudes. Its
   scaling, the difference from the maximum and a cache scale round 4 more times, each at most u of what Q bounds: a score is off by at
   most (2 D + 4) u Q, which is the relative error of exp; exp2 adds 2 u. Scores change only through their differences, so
   each p is off by at most E = 2 (2 D + 4) u Q + 4 u, the rounded maxima included.
 - The sum and the weighted sum have n terms each, in any order, with one rescaling a tile: 2 (2 n) u between them, 8 u for joining parts and dividing.
 - Prompts: p is rounded to the type of v, e(t), and the rounded p are summed too: o' - o = sum_j p_j d_j (v_j - o) / sum_j p_j (1 + d_j)
   with |d| <= e(t), at most e(t) (A + |o|) to first order. f16 reaches down to 2^-24 only: up to 2^-25 more for each p, where one of
   them is at least 1: 2^-25 (sum_j |v_j| + n |o|). One token, and bf16 prompts with f16 outputs: p is held in two pieces of the type,
   (2^-8)^2 at most, f16's down to 2^-24.
 - o is stored with one rounding, e(out), and f16 subnormals 2^-25.

    |o - o_ref| <= e(out) |o_ref| + 1.01 (2 E + (4 n + 8) u) A + 1.01 e_p (A + |o_ref|) + (f16: 1.01 2^-25 (sum_j |v_j| + n |o_ref|)) + 2^-25
"""
import math

import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
from test_kv_cache import _paged_copy

F16, BF16, U8, F32, I32, I64 = torch.float16, torch.bfloat16, torch.uint8, torch.float32, torch.int32, torch.int64
TYPES = {"f16": F16, "bf16": BF16}
U = 2.0 ** -24
E = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
FAKE = 0x100000000   # aligned, never dereferenced: a check fails first or there is nothing to do
BIG = 1 << 30


def _decode(**kw):
    a = dict(q=FAKE, ldq=6144, hsq=128, type=1, kc=FAKE + (1 << 24), vc=FAKE + (2 << 24), ks=FAKE + (3 << 24), vs=FAKE + (4 << 24), pages=9, page=16,
             table=FAKE + (5 << 24), width=3, lens=FAKE + (6 << 24), B=2, Hq=48, Hkv=8, D=128, scale=0.1, o=FAKE + (7 << 24), ot=0,
             ws=FAKE + (8 << 24), wsb=BIG, s=None)
    a.update(kw)
    return pq.lib().pq_attn_decode(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -2), (dict(width=-1), -2), (dict(type=2), -2), (dict(ot=2), -2), (dict(D=80), -2), (dict(Hq=0), -2), (dict(Hkv=0), -2), (dict(Hq=50), -2),
    (dict(Hq=65544), -2), (dict(scale=0.0), -2), (dict(scale=-1.0), -2), (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2),
    (dict(page=48), -2), (dict(pages=-1), -2), (dict(ldq=6148), -2), (dict(hsq=4), -2), (dict(ldq=-8), -2),
    (dict(q=None), -1), (dict(o=None), -1), (dict(lens=None), -1), (dict(table=None), -1), (dict(ks=None), -1), (dict(vc=None), -1),
    (dict(q=FAKE + 2), -3), (dict(o=FAKE + 8), -3), (dict(lens=FAKE + 2), -3), (dict(table=FAKE + 2), -3), (dict(kc=FAKE + 8), -3),
    (dict(B=2**31 - 1), -2), (dict(B=0), 0), (dict(B=0, q=None, o=None, ws=None, wsb=0), 0), (dict(scale=2.0**65), -2), (dict(scale=3e38), -2),
    (dict(o=FAKE), -2), (dict(o=FAKE + (1 << 24) + 16), -2), (dict(o=FAKE + (4 << 24)), -2), (dict(o=FAKE + (6 << 24)), -2), (dict(o=FAKE + (8 << 24)), -2),
    (dict(ws=FAKE + (1 << 24)), -2), (dict(o=FAKE + 2 * (6144 + 47 * 128 + 128) - 16), -2), (dict(pages=2**31 - 1, page=1024), -2),
])
def test_decode_refusals(kw, code):
    assert _decode(**kw) == code
    assert bool(pq.lib().pq_last_error()) == (code != 0)


def _prefill(**kw):
    a = dict(q=FAKE, ldq=8192, hsq=128, k=FAKE + (1 << 24), ldk=8192, hsk=128, v=FAKE + (2 << 24), ldv=8192, hsv=128, type=1, cu_q=FAKE + (3 << 24),
             cu_k=FAKE + (4 << 24), B=2, Tq=40, Tk=40, Hq=48, Hkv=8, D=128, scale=0.1, causal=1, o=FAKE + (5 << 24), ot=0, ws=FAKE + (6 << 24),
             wsb=BIG, s=None)
    a.update(kw)
    return pq.lib().pq_attn_prefill(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), -2), (dict(Tq=-1), -2), (dict(Tk=-1), -2), (dict(type=2), -2), (dict(ot=3), -2), (dict(D=192), -2), (dict(Hq=12), -2), (dict(Hkv=-8), -2),
    (dict(scale=0.0), -2), (dict(scale=float("nan")), -2), (dict(ldq=8196), -2), (dict(hsk=2), -2), (dict(ldv=-8), -2), (dict(ldk=2**31), -2),
    (dict(q=None), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(o=None), -1), (dict(cu_q=None), -1), (dict(cu_k=None), -1),
    (dict(q=FAKE + 8), -3), (dict(k=FAKE + 2), -3), (dict(v=FAKE + 4), -3), (dict(o=FAKE + 8), -3), (dict(cu_q=FAKE + 1), -3),
    (dict(Tq=2**31 - 1), -2), (dict(Tq=0), 0), (dict(B=0), 0), (dict(Tq=0, q=None, o=None), 0), (dict(scale=2.0**65), -2),
    (dict(o=FAKE), -2), (dict(o=FAKE + (1 << 24) + 16), -2), (dict(o=FAKE + (2 << 24) - 16), -2), (dict(o=FAKE + (3 << 24)), -2), (dict(o=FAKE + (4 << 24)), -2),
    (dict(Tk=2000, ws=FAKE + (2 << 24) + 16), -2), (dict(Tk=2000, ws=FAKE + (5 << 24)), -2),
    (dict(Tk=2**30 + 1, ldk=0, ldv=0), -2), (dict(Tq=2**30 + 1, Hq=1, Hkv=1, ldq=0), -2),
])
def test_prefill_refusals(kw, code):
    assert _prefill(**kw) == code
    assert bool(pq.lib().pq_last_error()) == (code != 0)


def _z(*shape, dtype=F16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,err", [
    (dict(q=_z(2, 16, 64)), ValueError), (dict(q=_z(2, 10, 128)), ValueError), (dict(q=_z(2, 2048)), ValueError), (dict(q=_z(2, 16, 128, dtype=F32)), TypeError),
    (dict(block_table=_z(3, 3, dtype=I32)), ValueError), (dict(block_table=_z(2, 3, dtype=I64)), TypeError), (dict(lengths=_z(3, dtype=I32)), ValueError),
    (dict(lengths=_z(2, dtype=I64)), TypeError), (dict(k_scale=None), ValueError), (dict(k_scale=None, v_scale=None), TypeError),
    (dict(out=_z(2, 16, 64)), ValueError), (dict(out=_z(2, 16, 128), dtype=BF16), TypeError), (dict(dtype=F32), TypeError),
    (dict(workspace=_z(4)), TypeError), (dict(k_cache=_z(3, 0, 16, 128, dtype=U8)), ValueError), (dict(), TypeError),
])
def test_decode_binding_refusals(kw, err):
    a = dict(q=_z(2, 16, 128), k_cache=_z(3, 8, 16, 128, dtype=U8), v_cache=_z(3, 8, 16, 128, dtype=U8), block_table=_z(2, 3, dtype=I32), lengths=_z(2, dtype=I32),
             k_scale=_z(3, 8, 16, dtype=F32), v_scale=_z(3, 8, 16, dtype=F32))
    a.update(kw)
    with pytest.raises(err):
        pq.attn_decode(**a)


@pytest.mark.parametrize("kw,err", [
    (dict(k=_z(4, 3, 128)), ValueError), (dict(k=_z(4, 2, 64)), ValueError), (dict(k=_z(4, 2, 128, dtype=BF16)), TypeError), (dict(v=_z(5, 2, 128)), ValueError),
    (dict(v=_z(4, 4, 128)), ValueError), (dict(q=_z(4, 128)), ValueError), (dict(cu_q=_z(0, dtype=I32)), ValueError), (dict(cu_q=_z(2, dtype=I64)), TypeError),
    (dict(cu_k=_z(3, dtype=I32)), ValueError), (dict(out=_z(3, 8, 128)), ValueError), (dict(out=_z(4, 8, 128), dtype=BF16), TypeError),
    (dict(q=_z(4, 128, 8).transpose(1, 2)), ValueError), (dict(workspace=_z(4)), TypeError), (dict(), TypeError),
])
def test_prefill_binding_refusals(kw, err):
    a = dict(q=_z(4, 8, 128), k=_z(4, 2, 128), v=_z(4, 2, 128), cu_q=_z(2, dtype=I32))
    a.update(kw)
    with pytest.raises(err):
        pq.attn_prefill(**a)


# ------------------------------------------------------------------------------------------
gpu = pytest.mark.gpu


def _reference(q, k, v, scale, visible):
    """q [R, D], k, v [n, D], visible [R, n] in 64 bits -> (o, Q, A, sum |v|); what is not visible is not read."""
    R, n = q.shape[0], k.shape[0]
    o, A, S, Q = torch.zeros_like(q), torch.zeros_like(q), torch.zeros_like(q), torch.zeros((R, 1), dtype=q.dtype, device=q.device)
    if n == 0:
        return o, Q, A, S
    a = (q @ k.t().contiguous() * scale).masked_fill(~visible, -math.inf)
    mag = (q.abs() @ k.abs().t().contiguous() * scale).masked_fill(~visible, 0)
    some = visible.any(-1, keepdim=True)
    p = torch.where(some, torch.softmax(torch.where(some, a, 0), -1), 0).masked_fill(~visible, 0)
    return p @ v, mag.amax(-1, keepdim=True), p @ v.abs(), visible.to(q.dtype) @ v.abs()


def _e_p(q, o):
    return 2.0 ** -16 if q.dtype == BF16 and o.dtype == F16 else E[q.dtype]


def _check(o, ref, n, D, dtype, e_p, what):
    want, Q, A, S = ref
    tol = E[o.dtype] * want.abs() + 1.01 * (2 * (2 * (2 * D + 4) * U * Q + 4 * U) + (4 * n + 8) * U) * A + 1.01 * e_p * (A + want.abs()) + 2.0 ** -25
    if dtype == F16:
        tol = tol + 1.01 * 2.0 ** -25 * (S + n * want.abs())
    err = (o.double() - want).abs()
    worst = float((err / tol).max()) if err.numel() else 0.0
    assert bool((err <= tol).all()), f"{what}: {worst:.2f} of the tolerance"
    return worst


def _heads(g, T, H, D, dtype, spread=0.3, device="cuda"):
    x = torch.randn((T, H, D), generator=g) * torch.exp(spread * torch.randn((T, H, 1), generator=g))
    return (x * torch.where(torch.rand((H, D), generator=g) < 1 / 16, 4.0, 1.0)).to(dtype).to(device)


def _cu(lens, first=0):
    return torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=I32, device="cuda")


def _prompts(g, lens, Hq, Hkv, D, dtype, ahead=0, behind=0):
    """The q, k and v columns of a merged projection; what stands before and behind the sequences is NaN."""
    T = ahead + sum(n for n, _ in lens) + behind
    Tk = ahead + sum(n for _, n in lens) + behind
    y = torch.full((T, (Hq + 2 * Hkv) * D), math.nan, dtype=dtype, device="cuda")
    z = torch.full((Tk, (Hq + 2 * Hkv) * D), math.nan, dtype=dtype, device="cuda")
    q = y[:, :Hq * D].unflatten(1, (Hq, D))
    k, v = z[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)), z[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    q[ahead:T - behind] = 0.7 * _heads(g, T - ahead - behind, Hq, D, dtype)
    k[ahead:Tk - behind] = _heads(g, Tk - ahead - behind, Hkv, D, dtype)
    v[ahead:Tk - behind] = _heads(g, Tk - ahead - behind, Hkv, D, dtype)
    return q, k, v, _cu([n for n, _ in lens], ahead), _cu([n for _, n in lens], ahead)


def _check_prompts(o, q, k, v, lens, ahead, causal, scale, what, hidden=None):
    """Every head of every sequence; hidden: the tolerance's reference sees nothing of these key rows."""
    Hq, D = q.shape[1:]
    G, at, kat, worst = Hq // k.shape[1], ahead, ahead, 0.0
    for b, (nq, nk) in enumerate(lens):
        visible = torch.ones((nq, nk), dtype=torch.bool, device="cuda")
        if causal:
            visible = visible.tril(nk - nq)
        for h in range(Hq):
            ks, vs = k[kat:kat + nk, h // G].double(), v[kat:kat + nk, h // G].double()
            ref = _reference(q[at:at + nq, h].double(), ks, vs, scale, visible)
            worst = max(worst, _check(o[at:at + nq, h], ref, nk, D, q.dtype, _e_p(q, o), f"{what}, sequence {b} ({nq}, {nk}), head {h}"))
        at, kat = at + nq, kat + nk
    return worst


SHAPES = [
    ([(1, 1)], 1, 1), ([(2, 2), (1, 1), (3, 3)], 2, 1), ([(37, 37)], 12, 12), ([(31, 31), (0, 0), (33, 33), (64, 64), (65, 65)], 6, 2),
    ([(127, 127), (1, 1), (129, 129), (300, 300)], 5, 1),
    ([(1, 513), (16, 100), (7, 7)], 8, 2),                        # chunks behind earlier keys
    ([(5, 3), (4, 0), (40, 8), (3, 5), (0, 9)], 4, 4),            # rows that see no key
    ([(200, 1000)], 16, 1), ([(513, 513)], 3, 3),
]


@gpu
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16"), ("f16", "bf16")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Hq,Hkv", SHAPES)
def test_prefill(lens, Hq, Hkv, D, kind, out, causal):
    g = torch.Generator().manual_seed(D + Hq + len(lens))
    ahead, behind = (3, 5) if len(lens) > 1 else (0, 0)
    q, k, v, cu_q, cu_k = _prompts(g, lens, Hq, Hkv, D, TYPES[kind], ahead, behind)
    o = torch.full((q.shape[0], Hq, D), 7.0, dtype=TYPES[out], device="cuda")
    same = all(a == b for a, b in lens)
    assert pq.attn_prefill(q, k, v, cu_q, None if same else cu_k, causal=causal, out=o) is o
    worst = _check_prompts(o, q, k, v, lens, ahead, causal, D ** -0.5, "prefill")
    assert bool((o[:ahead] == 7).all()) and bool((o[o.shape[0] - behind:] == 7).all())     # rows of no sequence
    made = pq.attn_prefill(q, k, v, cu_q, cu_k, causal=causal, dtype=TYPES[out])
    assert torch.equal(made[ahead:made.shape[0] - behind], o[ahead:o.shape[0] - behind])      # the same call, the same bits
    print(f"worst {worst:.2f} of the tolerance")


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,Hq,Hkv", [(2048, 2, 1), (1111, 6, 1)])
def test_prefill_long(T, Hq, Hkv, D):
    g = torch.Generator().manual_seed(T)
    q, k, v, cu, _ = _prompts(g, [(T, T)], Hq, Hkv, D, BF16)
    _check_prompts(pq.attn_prefill(q, k, v, cu), q, k, v, [(T, T)], 0, True, D ** -0.5, "long")


@gpu
@pytest.mark.parametrize("nq,nk", [(1, 20001), (33, 9000), (150, 6000)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_few_rows_behind_many_keys(nq, nk, D):
    g = torch.Generator().manual_seed(nq + D)
    lens = [(nq, nk), (3, 40), (1, 700)]
    q, k, v, cu_q, cu_k = _prompts(g, lens, 6, 1, D, BF16)
    _check_prompts(pq.attn_prefill(q, k, v, cu_q, cu_k), q, k, v, lens, 0, True, D ** -0.5, "few rows")


@gpu
@pytest.mark.parametrize("B,Hq,longest", [(100, 1, 3000), (150, 2, 2500), (65, 6, 1300), (300, 1, 60)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_prefill_of_many_sequences(B, Hq, longest, D):
    """More sequences than a wave has lanes, empty ones among them, some with their key tiles cut and some whole."""
    g = torch.Generator().manual_seed(B + D)
    nq = torch.randint(0, 6, (B,), generator=g).tolist()
    lens = [(n, n + int(longest * float(torch.rand((), generator=g)) ** 4)) for n in nq[:-2]] + [(140, 140 + longest), (0, 9)]
    q, k, v, cu_q, cu_k = _prompts(g, lens, Hq, 1, D, BF16)
    _check_prompts(pq.attn_prefill(q, k, v, cu_q, cu_k), q, k, v, lens, 0, True, D ** -0.5, "many sequences")


@gpu
@pytest.mark.parametrize("scale", [1e-4, 0.02, 1.0, 30.0])
def test_prefill_scales(scale):
    """From weights that hardly differ to one that takes all; scores whose maximum rises and falls along the keys."""
    g = torch.Generator().manual_seed(3)
    T, D = 300, 64
    q, k, v, cu, _ = _prompts(g, [(T, T)], 2, 1, D, F16)
    ramp = torch.cat([torch.linspace(-3, 3, T // 2), torch.linspace(3, -3, T - T // 2)]).cuda()
    k += (ramp[:, None, None] * 0.3).half()
    q += 0.5
    _check_prompts(pq.attn_prefill(q, k, v, cu, scale=scale), q, k, v, [(T, T)], 0, True, float(np.float32(scale)), "scales")


@gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_prefill_values_that_a_query_does_not_see(kind, D, bad):
    """Infinities and NaN in later keys and values, and in the neighbouring sequences, change no earlier query."""
    g = torch.Generator().manual_seed(9)
    lens, at = [(70, 70), (150, 150), (40, 40)], 100      # row 100 of the second sequence
    q, k, v, cu, _ = _prompts(g, lens, 4, 2, D, TYPES[kind])
    clean = pq.attn_prefill(q, k, v, cu)
    k2, v2 = k.clone(), v.clone()
    v2[70 + at, 0, 5], k2[70 + at, 1] = bad, bad
    k2[220 + 39], v2[220 + 39] = bad, bad                  # the last row of all
    o = pq.attn_prefill(q, k2, v2, cu)
    assert bool(torch.isfinite(o[:70 + at]).all()) and bool(torch.isfinite(o[220:220 + 39]).all())
    # heads 0, 1 see the bad value in one channel only, from row `at` on
    seen = o[70 + at:220, :2]
    assert not bool(torch.isfinite(seen[:, :, 5]).any()) and bool(torch.isfinite(seen[:, :, :5]).all()) and bool(torch.isfinite(seen[:, :, 6:]).all())
    if math.isinf(bad):
        weight = clean[70 + at:220, :2, 5].isfinite()
        assert bool((seen[:, :, 5][weight].float() == bad).all() | torch.isnan(seen[:, :, 5]).any())
    lens2, sane = [(70, 70), (at, at)], slice(0, 70 + at)
    _check_prompts(o[sane], q[sane], k[sane], v[sane], lens2, 0, True, D ** -0.5, "unseen")


@gpu
@pytest.mark.parametrize("nk", [70, 3000])
def test_prefill_queries_that_are_not_finite(nk):
    """NaN and infinities in a query make its own row NaN, and no other one."""
    g = torch.Generator().manual_seed(12)
    lens = [(70, nk), (40, 40)]
    q, k, v, cu_q, cu_k = _prompts(g, lens, 2, 1, 128, BF16)
    q[5, 0, 7], q[33, 1, 0], q[64] = math.nan, math.inf, -math.inf
    o = pq.attn_prefill(q, k, v, cu_q, cu_k)
    bad = torch.zeros(o.shape[:2], dtype=torch.bool, device="cuda")
    bad[5, 0] = bad[33, 1] = bad[64, 0] = bad[64, 1] = True
    assert bool(torch.isnan(o[bad]).all()) and bool(torch.isfinite(o[~bad]).all())
    # the others within their tolerance (their last bits may differ: rows of a wave raise what their weights are taken against together)
    at = kat = 0
    for nq, n in lens:
        visible = torch.ones((nq, n), dtype=torch.bool, device="cuda").tril(n - nq)
        for h in range(2):
            good = ~bad[at:at + nq, h]
            ref = _reference(q[at:at + nq, h][good].double(), k[kat:kat + n, 0].double(), v[kat:kat + n, 0].double(), 128 ** -0.5, visible[good])
            _check(o[at:at + nq, h][good], ref, n, 128, BF16, E[BF16], f"beside queries that are not finite, head {h}")
        at, kat = at + nq, kat + n


@gpu
def test_prefill_largest_values():
    """Values that a weight above 1 would carry past binary32, and scores whose maximum keeps rising along the keys."""
    g = torch.Generator().manual_seed(13)
    T, D = 200, 64
    q, k, v, cu, _ = _prompts(g, [(T, T)], 2, 1, D, BF16)
    v *= 1e36
    k[:, 0, 0] = torch.linspace(-40, 40, T, device="cuda")
    q[:, :, 0] = 30
    _check_prompts(pq.attn_prefill(q, k, v, cu), q, k, v, [(T, T)], 0, True, D ** -0.5, "largest values")


@gpu
def test_prefill_non_causal_infinite_values():
    """With every key seen, an infinite value gives infinities in its channel wherever its weight is not zero, and no NaN."""
    g = torch.Generator().manual_seed(2)
    q, k, v, cu, _ = _prompts(g, [(45, 45)], 2, 1, 128, BF16)
    v[44, 0, 3], v[7, 0, 100] = math.inf, -math.inf
    o = pq.attn_prefill(q, k, v, cu, causal=False)
    assert bool((o[:, :, 3] == math.inf).all()) and bool((o[:, :, 100] == -math.inf).all())
    rest = [c for c in range(128) if c not in (3, 100)]
    assert bool(torch.isfinite(o[:, :, rest]).all())


@gpu
def test_prefill_lengths_that_pass_the_rows():
    """Boundaries past the tensors count as their ends: nothing outside is read or written."""
    g = torch.Generator().manual_seed(2)
    q, k, v, _, _ = _prompts(g, [(40, 40)], 2, 1, 64, BF16)
    whole = torch.full((48, 2, 64), 7.0, dtype=BF16, device="cuda")
    pq.attn_prefill(q, k, v, torch.tensor([0, 1000], dtype=I32, device="cuda"), out=whole[:40])
    _check_prompts(whole[:40], q, k, v, [(40, 40)], 0, True, 0.125, "past the end")
    assert bool((whole[40:] == 7).all())
    o = torch.full((40, 2, 64), 7.0, dtype=BF16, device="cuda")
    pq.attn_prefill(q, k, v, torch.tensor([0, 20, 10], dtype=I32, device="cuda"), torch.tensor([5, -3, 2 ** 31 - 1], dtype=I32, device="cuda"), out=o)
    torch.cuda.synchronize()
    assert bool((o[20:] == 7).all())


# ------------------------------------------------------------------------------------------
def _check_decode(o, q, rows, lens, scale, what, quant=False):
    Hq, D = q.shape[1:]
    worst = 0.0
    for b, n in enumerate(lens):
        ks, vs = (torch.as_tensor(r[b]).cuda() for r in rows)
        G = Hq // ks.shape[1]
        for h in range(ks.shape[1]):
            qs = q[b, h * G:(h + 1) * G].double()
            ref = _reference(qs, ks[:, h].contiguous(), vs[:, h].contiguous(), scale, torch.ones((G, n), dtype=torch.bool, device="cuda"))
            worst = max(worst, _check(o[b, h * G:(h + 1) * G], ref, n, D, q.dtype, 2.0 ** -16, f"{what}, sequence {b} ({n}), key head {h}"))
    return worst


DECODE = [
    ([1], 1, 1, 16), ([0], 2, 2, 16), ([2, 0, 15, 16, 17, 31, 32, 33, 63, 64, 65], 6, 2, 16), ([127, 128, 129, 300, 1], 8, 8, 32),
    ([1000, 3, 700], 16, 1, 64), ([513, 2049], 24, 4, 16), ([255, 256, 257], 17, 1, 256), ([40, 1025], 48, 1, 1024), ([5000], 12, 2, 128),
    ([1] * 70 + [90], 5, 5, 16),
]


@gpu
@pytest.mark.parametrize("kind,cache,out", [("bf16", "e4m3", "f16"), ("f16", "e4m3", "f16"), ("bf16", "bf16", "bf16"), ("f16", "f16", "f16"), ("f16", "e4m3", "bf16")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("lens,Hq,Hkv,page", DECODE)
def test_decode(lens, Hq, Hkv, page, D, kind, cache, out):
    g = torch.Generator().manual_seed(sum(lens) + D)
    caches, scales, table, rows = _paged_copy(g, lens, Hkv, page, D, cache)
    q = _heads(g, len(lens), Hq + 1, D, TYPES[kind])[:, 1:]          # rows apart
    dev = [c.cuda() for c in caches] + [table.cuda(), torch.tensor(lens, dtype=I32, device="cuda")] + [None if s is None else s.cuda() for s in scales]
    o = torch.full((len(lens), Hq, D), 7.0, dtype=TYPES[out], device="cuda")
    assert pq.attn_decode(q, *dev, out=o) is o
    worst = _check_decode(o, q, rows, lens, D ** -0.5, "decode")
    assert torch.equal(pq.attn_decode(q, *dev, dtype=TYPES[out]), o)
    print(f"worst {worst:.2f} of the tolerance")


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "bf16"])
@pytest.mark.parametrize("lens,Hq,Hkv,page,D", [([70001], 6, 1, 16, 128), ([30000, 0, 1, 9000, 17], 8, 2, 64, 64), ([20011, 20012], 4, 2, 32, 256)])
def test_decode_long(lens, Hq, Hkv, page, D, cache):
    g = torch.Generator().manual_seed(sum(lens))
    caches, scales, table, rows = _paged_copy(g, lens, Hkv, page, D, cache)
    q = _heads(g, len(lens), Hq, D, BF16)
    dev = [c.cuda() for c in caches] + [table.cuda(), torch.tensor(lens, dtype=I32, device="cuda")] + [None if s is None else s.cuda() for s in scales]
    _check_decode(pq.attn_decode(q, *dev, dtype=F16), q, rows, lens, D ** -0.5, "long")


@gpu
@pytest.mark.parametrize("cache", ["e4m3", "f16"])
def test_decode_pages_that_are_not_the_caches(cache):
    """A position whose page number is not the cache's is left out; lengths end at the table's width; negative ones are 0."""
    g = torch.Generator().manual_seed(4)
    lens, page, D = [100, 60, 50], 16, 64
    caches, scales, table, rows = _paged_copy(g, lens, 2, page, D, cache)
    bad = table.clone()
    bad[0, 2], bad[1, 0], bad[1, 1], bad[1, 2], bad[1, 3] = caches[0].shape[0], -1, -2 ** 31, 2 ** 31 - 1, caches[0].shape[0]
    keep = [[i for i in range(100) if not 32 <= i < 48], [], []]
    q = _heads(g, 3, 4, D, F16)
    asked = torch.tensor([100, 60, -5], dtype=I32, device="cuda")
    dev = [c.cuda() for c in caches]
    sc = [None if s is None else s.cuda() for s in scales]
    o = pq.attn_decode(q, *dev, bad.cuda(), asked, *sc)
    kept = [[r[b][keep[b]] for b in range(3)] for r in rows]
    _check_decode(o, q, kept, [len(x) for x in keep], D ** -0.5, "bad pages")
    assert bool((o[1:] == 0).all())
    narrow = table[:, :2].contiguous().cuda()
    o = pq.attn_decode(q, *dev, narrow, torch.tensor([100, 2 ** 31 - 1, 20], dtype=I32, device="cuda"), *sc)
    _check_decode(o, q, [[r[0][:32], r[1][:32], r[2][:20]] for r in rows], [32, 32, 20], D ** -0.5, "narrow table")
    o = pq.attn_decode(q, *dev, table[:, :0].contiguous().cuda(), asked, *sc)
    assert bool((o == 0).all())


@gpu
@pytest.mark.parametrize("scale", [1e-4, 0.125, 4.0, 30.0])
@pytest.mark.parametrize("cache", ["e4m3", "f16"])
def test_decode_scales(scale, cache):
    g = torch.Generator().manual_seed(6)
    lens, D = [400, 37], 64
    caches, scales, table, rows = _paged_copy(g, lens, 1, 16, D, cache)
    q = _heads(g, 2, 16, D, F16)
    sc = [None if s is None else s.cuda() for s in scales]
    o = pq.attn_decode(q, *(c.cuda() for c in caches), table.cuda(), torch.tensor(lens, dtype=I32, device="cuda"), *sc, scale=scale)
    _check_decode(o, q, rows, lens, float(np.float32(scale)), "scales")


@gpu
def test_decode_values_that_are_not_finite():
    """A visible NaN or infinity reaches its own sequence and head only."""
    g = torch.Generator().manual_seed(8)
    lens, D = [70, 33], 128
    caches, _, table, rows = _paged_copy(g, lens, 2, 16, D, "bf16")
    caches[1][table[0, 1], 1, 3, 9] = math.inf
    q = _heads(g, 2, 4, D, BF16)
    o = pq.attn_decode(q, *(c.cuda() for c in caches), table.cuda(), torch.tensor(lens, dtype=I32, device="cuda"))
    assert bool(torch.isfinite(o[1]).all()) and bool(torch.isfinite(o[0, :2]).all())
    assert not bool(torch.isfinite(o[0, 2:, 9]).any()) and bool(torch.isfinite(o[0, 2:, :9]).all()) and bool(torch.isfinite(o[0, 2:, 10:]).all())


@gpu
def test_one_token_and_a_prompt_of_one_row_agree():
    """attn_prefill of one row behind nk - 1 keys is attn_decode of the same keys in a 16-bit cache, within both tolerances."""
    g = torch.Generator().manual_seed(11)
    n, Hq, Hkv, D, page = 333, 12, 2, 128, 16
    caches, _, table, rows = _paged_copy(g, [n], Hkv, page, D, "bf16")
    q = _heads(g, 1, Hq, D, BF16)
    k, v = (r[0].to(BF16).cuda() for r in rows)
    a = pq.attn_decode(q, *(c.cuda() for c in caches), table.cuda(), torch.tensor([n], dtype=I32, device="cuda"))
    b = pq.attn_prefill(q, k, v, _cu([1]), _cu([n]))
    for h in range(Hq):
        ref = _reference(q[0, h:h + 1].double(), k[:, h // 6].double(), v[:, h // 6].double(), D ** -0.5, torch.ones((1, n), dtype=torch.bool, device="cuda"))
        _check(a[0, h:h + 1], ref, n, D, BF16, 2.0 ** -16, "decode")
        _check(b[0, h:h + 1], ref, n, D, BF16, 2.0 ** -8, "prefill")
