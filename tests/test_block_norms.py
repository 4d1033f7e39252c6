"""pq_block_norms: refusals (CPU) and parity with the formula in 64 bits (GPU).

    n = x rstd(x) w_post',  h = fl(res_scale res + scale a(gate) n),  hs = fl(h rstd(h) w_pre')

Tolerance, with u = 2^-24 and e = eps/2 of the stored type. The sum of K squares has at most 32
terms per thread, 6 wave and 15 workgroup additions, so its relative error is at most 55 u; rstd halves it
and adds the mean's division, the eps, the square root and the division (4 u): 32 u. Products with x, w' (one
rounding for 1 + w), the gate and the scale: 6 u; the gate's own function at most 8 u (exp2 and the reciprocal
within 1 ulp; the tangent's series 4.5 u, its quotient 7.9 u) and, for the sigmoid, 2 |t| u more: its exponent -t log2(e) is a rounded product
with a rounded constant, and a relative u of the exponent is |t| u of exp(-t). So |n-part| <= (48 + 2 |t|) u relative, the
residual's product 1 u, their sum 1 u:

    |h - h_ref|   <= e |h_ref|  + 1.01 ((50 + 2 |t|) u |scale a n| + 3 u |res_scale res|) + tiny      (2 |t|: sigmoid gates)
    |hs - hs_ref| <= e |hs_ref| + 1.01 * 48 u |hs_ref| + tiny          (hs_ref from the kernel's own stored h)

tiny: half the smallest subnormal of the stored type (f32: the smallest normal, as intermediates may flush)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq

U = 2.0 ** -24
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126, torch.float32: 2.0 ** -126}
FAKE = 0x100000000   # aligned, never dereferenced: a check fails first or M == 0


def _call(**kw):
    a = dict(x=FAKE, ldx=256, xt=1, res=FAKE + (1 << 20), ldr=256, rt=0, wpost=FAKE + (2 << 20), gate=None, ldg=0, gc=256,
             ga=0, wpre=FAKE + (3 << 20), eps=1e-6, scale=1.0, rscale=1.0, gemma=0, M=4, K=256, ro=FAKE + (4 << 20), ldo=256,
             hs=FAKE + (5 << 20), ldh=256, ot=0, s=None)
    a.update(kw)
    return pq.lib().pq_block_norms(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -2), (dict(K=0), -2), (dict(K=12), -2), (dict(K=32776, ldx=40000, ldr=40000, ldo=40000, ldh=40000), -2),
    (dict(xt=2), -2), (dict(xt=3), -2), (dict(rt=3), -2), (dict(ot=2), -2), (dict(ga=3), -2),
    (dict(eps=0.0), -2), (dict(eps=float("nan")), -2), (dict(eps=float("inf")), -2), (dict(eps=-1e-6), -2),
    (dict(ldx=248), -2), (dict(ldx=260), -2), (dict(ldr=260), -2), (dict(ldo=128), -2), (dict(ldh=252), -2),
    (dict(rt=2, ldr=258), -2), (dict(gate=FAKE + (6 << 20), gc=2), -2), (dict(gate=FAKE + (6 << 20), ldg=-8), -2),
    (dict(gate=FAKE + (6 << 20), ldg=128), -2), (dict(gate=FAKE + (6 << 20), ldg=260), -2),
    (dict(x=None), -1), (dict(res=None), -1), (dict(ro=None), -1), (dict(hs=None), -1),
    (dict(x=FAKE + 8), -3), (dict(res=FAKE + (1 << 20) + 2), -3), (dict(wpost=FAKE + (2 << 20) + 8), -3), (dict(hs=FAKE + (5 << 20) + 4), -3),
    (dict(gate=FAKE + (6 << 20) + 2), -3), (dict(gate=FAKE + (6 << 20) + 1, gc=1, ldg=1), -3),
    # an output over an input, or over the other output
    (dict(ro=FAKE), -2), (dict(hs=FAKE), -2), (dict(hs=FAKE + (1 << 20)), -2), (dict(hs=FAKE + (4 << 20)), -2),
    (dict(ro=FAKE + (1 << 20) + 512), -2),                       # the residual shifted by one row
    (dict(ro=FAKE + (1 << 20), ldo=512), -2),                    # the residual with another stride
    (dict(hs=FAKE + (3 << 20) - 512), -2), (dict(gate=FAKE + (4 << 20), ldg=0), -2),
    (dict(M=2**31 - 1), -2), (dict(M=2**26 + 2**10, K=8, ldx=8, ldr=8, ldo=8, ldh=8, gc=8), -2),
    (dict(M=0), 0), (dict(M=0, x=None, hs=None), 0), (dict(M=0, K=32768, ldx=32768, ldr=32768, ldo=32768, ldh=32768), 0),
])
def test_refusals(kw, code):
    assert _call(**kw) == code
    assert bool(pq.lib().pq_last_error()) == (code != 0)


def _t(*shape, dtype=torch.float16):
    return torch.zeros(shape, dtype=dtype)


@pytest.mark.parametrize("kw,err", [
    (dict(x=_t(4, 256, dtype=torch.float32)), TypeError), (dict(x=_t(256)), ValueError),
    (dict(residual=_t(4, 256, dtype=torch.float64)), TypeError), (dict(residual=_t(3, 256)), ValueError), (dict(residual=None), TypeError),
    (dict(w_pre=_t(128)), ValueError), (dict(w_pre=_t(256), w_post=_t(256, dtype=torch.bfloat16)), TypeError),
    (dict(w_pre=_t(256, dtype=torch.float32)), TypeError), (dict(gate=_t(3, 256)), ValueError), (dict(gate=_t(128)), ValueError),
    (dict(gate=_t(4, 256, dtype=torch.bfloat16)), TypeError), (dict(gate=_t(3, 1)), ValueError), (dict(gate_act="silu"), ValueError),
    (dict(out=_t(4, 256)), ValueError), (dict(w_pre=_t(256), out=_t(4, 128)), ValueError), (dict(residual_out=_t(4, 256, dtype=torch.float32)), TypeError),
    (dict(x=_t(256, 4).t()), ValueError), (dict(), TypeError),   # the last: CPU tensors
])
def test_binding_refusals(kw, err):
    a = dict(x=_t(4, 256), residual=_t(4, 256))
    a.update(kw)
    with pytest.raises(err):
        pq.block_norms(a.pop("x"), a.pop("residual"), **a)


# ------------------------------------------------------------------------------------------
gpu = pytest.mark.gpu


def _norm(v, w, eps, gemma):
    f = v.double()
    return f / torch.sqrt((f * f).mean(-1, keepdim=True) + eps) * (w.double() + (1.0 if gemma else 0.0))


def _act(t, act):
    t = t.double()
    return torch.sigmoid(t) if act == "sigmoid" else torch.tanh(t) if act == "tanh" else t


def _reference(x, res, w_post, gate, eps, scale, res_scale, gate_act, gemma):
    """(h_ref in 64 bits, (1 + 2 |t| / 50) |scale a n|, |res_scale res|)"""
    n = _norm(x, w_post, eps, gemma) if w_post is not None else x.double()
    more = 1.0
    if gate is not None:
        n = n * _act(gate, gate_act)
        more = 1 + gate.double().abs() / 25 if gate_act == "sigmoid" else 1.0
    n, r = np.float32(scale).item() * n, np.float32(res_scale).item() * res.double()
    return n + r, n.abs() * more, r.abs()


def _check(tag, got, ref_parts, w_pre, eps, gemma):
    h, hs = got
    h_ref, mag_n, mag_r = ref_parts
    e = torch.finfo(h.dtype).eps / 2
    bound = e * h_ref.abs() + 1.01 * (50 * U * mag_n + 3 * U * mag_r) + TINY[h.dtype]
    ratio = ((h.double() - h_ref).abs() / bound).max().item() if h.numel() else 0.0
    ratio2 = 0.0
    if hs is not None and hs.numel():
        hs_ref = _norm(h, w_pre, eps, gemma)
        e = torch.finfo(hs.dtype).eps / 2
        bound = (e + 1.01 * 48 * U) * hs_ref.abs() + TINY[hs.dtype]
        ratio2 = ((hs.double() - hs_ref).abs() / bound).max().item()
    print(f"[norms {tag}] worst error/bound: h {ratio:.3f}, hs {ratio2:.3f}", flush=True)
    assert ratio <= 1.0 and ratio2 <= 1.0, tag


def _inputs(M, K, xt, rt, ot, gate, seed, post=True, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rows(cols, dtype, size):
        step = 8 * ((cols + 7) // 8) + pad
        buf = (size * torch.randn((M, step), generator=g, device="cuda")).to(dtype)
        return buf[:, :cols]
    x, res = rows(K, xt, 2.0), rows(K, rt, 4.0)
    w = (1 + 0.3 * torch.randn((2, K), generator=g, device="cuda")).to(ot)
    gt = None if gate is None else (rows(K, xt, 1.0) if gate == "rows" else
                                    rows(1, xt, 1.0) if gate == "token" else rows(K, xt, 1.0)[0].clone())
    return x, res, (w[0].contiguous() if post else None), gt, w[1].contiguous()


@gpu
@pytest.mark.parametrize("xt,rt,ot", list(itertools.product(("f16", "bf16"), ("f16", "bf16", "f32"), ("f16", "bf16"))))
def test_types(xt, rt, ot):
    for i, (gate, act, gemma) in enumerate([(None, "none", True), ("rows", "sigmoid", False), ("channel", "none", False), ("token", "tanh", True)]):
        M, K = (5, 640) if i % 2 else (3, 1000)
        x, res, wp, gt, wn = _inputs(M, K, TYPES[xt], TYPES[rt], TYPES[ot], gate, 10 + i)
        print(f"[norms types] {xt} {rt} {ot} gate={gate} {act}", flush=True)
        got = pq.block_norms(x, res, w_post=wp, gate=gt, w_pre=wn, eps=1e-5, scale=0.22, res_scale=0.5, gate_act=act, gemma=gemma)
        _check(f"{xt} {rt} {ot} {gate}", got, _reference(x, res, wp, gt, 1e-5, 0.22, 0.5, act, gemma), wn, 1e-5, gemma)


@gpu
@pytest.mark.parametrize("M,K", [(1, 8), (2, 16), (1, 504), (1, 512), (3, 520), (7, 4096), (5, 4104), (2, 8192), (3, 8200),
                                 (2, 16384), (2, 18432), (2, 32768), (1, 5120), (257, 5120), (1025, 1024)])
@pytest.mark.parametrize("rt", ["f16", "f32"])
def test_sizes(M, K, rt):
    x, res, wp, gt, wn = _inputs(M, K, torch.bfloat16, TYPES[rt], torch.float16, "rows", M + K, pad=8)
    print(f"[norms sizes] M={M} K={K} {rt}", flush=True)
    h = torch.full((M + 2, K + 16), 7.0, dtype=TYPES[rt], device="cuda")
    hs = torch.full((M + 2, K + 8), 7.0, dtype=torch.float16, device="cuda")
    got = pq.block_norms(x, res, w_post=wp, gate=gt, w_pre=wn, residual_out=h[:M, :K], out=hs[:M, :K])
    _check(f"M={M} K={K} {rt}", got, _reference(x, res, wp, gt, 1e-6, 1.0, 1.0, "none", False), wn, 1e-6, False)
    assert torch.all(h[M:] == 7) and torch.all(h[:, K:] == 7) and torch.all(hs[M:] == 7) and torch.all(hs[:, K:] == 7)


@gpu
def test_parts_left_out():
    """Without the post-norm, without the pre-norm, without either; a gate row or value shared by every token."""
    x, res, wp, gt, wn = _inputs(6, 384, torch.float16, torch.float16, torch.float16, "rows", 3)
    for post, pre in itertools.product((True, False), repeat=2):
        got = pq.block_norms(x, res, w_post=wp if post else None, gate=gt, w_pre=wn if pre else None, gate_act="sigmoid")
        assert (got[1] is None) == (not pre)
        _check(f"post={post} pre={pre}", got, _reference(x, res, wp if post else None, gt, 1e-6, 1.0, 1.0, "sigmoid", False), wn, 1e-6, False)
    a = pq.block_norms(x, res, wp, gt[1].expand(6, 384), wn)
    b = pq.block_norms(x, res, wp, gt[1].clone(), wn)
    c = pq.block_norms(x, res, wp, gt[1].repeat(6, 1), wn)
    one = torch.full((1, 1), 0.75, dtype=torch.float16, device="cuda")
    d = pq.block_norms(x, res, wp, one.expand(6, 1), wn)
    e = pq.block_norms(x, res, wp, torch.full((6, 384), 0.75, dtype=torch.float16, device="cuda"), wn)
    for p, q in ((a, b), (a, c), (d, e)):
        assert torch.equal(p[0], q[0]) and torch.equal(p[1], q[1])


@gpu
@pytest.mark.parametrize("M,K,rt", [(1, 5120, "f16"), (9, 5120, "f32"), (70, 16392, "bf16")])
def test_in_place_and_halves_of_one_buffer(M, K, rt):
    x, res, wp, gt, wn = _inputs(M, K, torch.bfloat16, TYPES[rt], torch.bfloat16, "channel", 5)
    h, hs = pq.block_norms(x, res, wp, gt, wn)
    again = res.contiguous().clone()
    buf = torch.empty((M, 2 * K), dtype=torch.bfloat16, device="cuda")
    h2, hs2 = pq.block_norms(x, again, wp, gt, wn, residual_out=again, out=buf[:, K:])
    assert h2.data_ptr() == again.data_ptr() and torch.equal(h, h2) and torch.equal(hs, hs2)
    if rt == "bf16":
        h3, hs3 = pq.block_norms(x, res, wp, gt, wn, residual_out=buf[:, :K], out=buf[:, K:])
        assert torch.equal(h, h3) and torch.equal(hs, hs3)
    with pytest.raises(pq.PQError):
        pq.block_norms(x, again, wp, gt, wn, residual_out=again, out=again if rt == "bf16" else again.view(torch.bfloat16)[:, :K])


@gpu
def test_zero_and_non_finite_rows():
    x, res, wp, gt, wn = _inputs(6, 1024, torch.bfloat16, torch.bfloat16, torch.bfloat16, "rows", 8)
    x[1], res[1] = 0, 0
    clean = pq.block_norms(x, res, wp, gt, wn)
    assert not clean[0][1].any() and not clean[1][1].any()
    x, res = x.clone(), res.clone()
    x[2, 5] = float("nan")
    x[3, 1000] = float("inf")
    res[4, 7] = float("-inf")
    h, hs = pq.block_norms(x, res, wp, gt, wn)
    for r in (0, 1, 5):
        assert torch.equal(h[r], clean[0][r]) and torch.equal(hs[r], clean[1][r])
    assert torch.isnan(h[2]).all() and torch.isnan(hs[2]).all()
    assert torch.isnan(h[3, 1000]) and torch.isnan(hs[3]).all()       # inf * rstd(inf) = inf * 0
    assert h[4, 7] == float("-inf") and torch.isnan(hs[4, 7]) and not hs[4, :7].any()


@gpu
def test_empty_and_streams_and_graph():
    x, res, wp, gt, wn = _inputs(33, 2048, torch.bfloat16, torch.float16, torch.float16, "rows", 9)
    h, hs = pq.block_norms(x[:0], res[:0], wp, gt[:0], wn)
    assert h.shape == (0, 2048) and hs.shape == (0, 2048)
    want = pq.block_norms(x, res, wp, gt, wn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pq.block_norms(x, res, wp, gt, wn, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    stream_h, out = torch.empty_like(res), torch.empty_like(res)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.block_norms(x, res, wp, gt, wn, residual_out=stream_h, out=out)
    for r in range(3):
        stream_h.zero_()
        out.zero_()
        x.mul_(0.5) if r == 1 else None
        g.replay()
        eager = pq.block_norms(x, res, wp, gt, wn)
        torch.cuda.synchronize()
        assert torch.equal(stream_h, eager[0]) and torch.equal(out, eager[1]), r


@gpu
@pytest.mark.parametrize("xt", [torch.float16, torch.bfloat16])
def test_gate_extremes(xt):
    """Gates at and past the ends of the functions, infinite and NaN: one value per element, per token and per channel."""
    vals = torch.tensor([0.0, -0.0, 1e-6, -0.3, 0.498, -0.5, 0.502, -20.0, 0.7, -80.0, 88.0, -88.0, 200.0, -200.0, 6e4, -6e4], device="cuda").to(xt)
    K = 256
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((16, K), generator=g, device="cuda").to(xt)
    res = torch.randn((16, K), generator=g, device="cuda")
    for act in ("sigmoid", "tanh"):
        for gate in (vals[:, None].expand(16, K).contiguous(), vals[:, None].contiguous(), vals.repeat(16)):
            got = pq.block_norms(x, res, gate=gate, gate_act=act)
            _check(f"extremes {act} {tuple(gate.shape)}", got, _reference(x, res, None, gate, 1e-6, 1.0, 1.0, act, False), None, 1e-6, False)
        gate = torch.zeros((16, K), dtype=xt, device="cuda")
        gate[0], gate[1], gate[2, 7] = float("inf"), float("-inf"), float("nan")
        h, _ = pq.block_norms(x, res, gate=gate, gate_act=act)
        assert torch.equal(h[0], res[0] + x[0].float()) and torch.equal(h[1], res[1] if act == "sigmoid" else res[1] - x[1].float())
        assert torch.isnan(h).sum() == 1 and torch.isnan(h[2, 7])


@gpu
def test_sigmoid_ends_with_the_normal_numbers():
    """(5 + 2 |t|) u of the sigmoid down to 2^-126, 0 below; with a stream of zeros nothing covers the gate's error. The product
    with x is exact (a power of two), the f32 stream rounds nothing."""
    gates = torch.tensor([-60.0, -80.0, -86.5, -87.0, -87.5, -88.0, -89.0, -104.0, -3e4], device="cuda").bfloat16()[:, None]
    x = torch.full((9, 8), 2.0 ** 10, device="cuda").bfloat16()
    for gate in (gates, gates.expand(9, 8).contiguous()):
        h, _ = pq.block_norms(x, torch.zeros((9, 8), device="cuda"), gate=gate, gate_act="sigmoid")
        t = gates[:4].double()
        ref = torch.sigmoid(t) * 2.0 ** 10
        assert ((h[:4].double() - ref).abs() <= (5 + 2 * t.abs()) * U * ref).all() and not h[4:].any()
