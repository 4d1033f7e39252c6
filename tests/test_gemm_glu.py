"""pq_gemm_glu: refusals (CPU) and parity with the formula in 64 bits (GPU).

    g = sum_k a W[:, :F],  u = sum_k a W[:, F:],  h = act(g) u,   a = asg D(code),  W = sc (c - 8) - fl16(sc (zp - 8))

Tolerance. g and u come from the GEMM's arithmetic (u24 = 2^-24, G groups). The matrix core multiplies exactly, aligns the 8
products of 8 neighbouring k to the largest exponent among them and drops what lies below 2^-13 of that power of two, toward
zero (measured: beside 448 * 15 = 1.64 * 2^12, exponents 8 and 3, a product of 2^-2 in the same 8 arrives and one of 2^-3 does
not; in other 8s all do). A code's e4m3 byte has the exponent of 8 to 15 whatever the code, so the dropped parts of a block are at most
7 * 2^-13 * 8 max|D|: X = sum asg sc (sum over blocks of 8 of max|D|) counts 7 * 2^-10. The blocks' sums and the fold add
g1 = (2*128 + G + 16) u24 of the sum of magnitudes Y = sum asg sc sum|D| c; the zero point as a product
of bf16 pieces or in binary32, g2 = 2^-14 + (3G + 16) u24 of Z = sum asg |rs| |8 sc + zsc|. E = 7 * 2^-10 X + g1 Y + g2 Z bounds either.
silu and gelu have slopes below 1.13 and |act(g)| <= |g|. act itself is g sigmoid(t), |t| <= 110 wherever sigmoid is a normal
number: t rounds by 4 u24 relative (the polynomial), t log2(e) once more, exp2, the sum, the reciprocal and two products by
8 u24: at most (5 * 110 + 8) u24 < 2^-14 of |h|; below that sigmoid < 2^-126 and h < 2^-118 |u|. So

    |h - h_ref| <= e |h_ref| + (1 + e) (1.13 Eg |u| + |act(g)| Eu + 1.13 Eg Eu + 2^-14 |h_ref| + 2^-118 |u|) + tiny

with e = eps/2 of h's type and tiny half its smallest subnormal (bf16: the smallest normal)."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
from oracle import awq

U24 = 2.0 ** -24
FAKE = 0x100000000
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _call(**kw):
    a = dict(a=FAKE, asg=FAKE, rs=FAKE, M=4, K=256, P=1, wpk=FAKE, sz=FAKE, F=64, act=0, h=FAKE, ldh=64, ht=0, ws=FAKE,
             ws_bytes=1 << 24, prepared=0, s=None)
    a.update(kw)
    return pq.lib().pq_gemm_glu(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -2), (dict(K=0), -2), (dict(K=100), -2), (dict(F=0), -2), (dict(F=24), -2), (dict(F=(1 << 23) + 16, ldh=1 << 24), -2),
    (dict(ldh=62), -2), (dict(ldh=65), -2), (dict(act=2), -2), (dict(act=-1), -2), (dict(ht=2), -2),
    (dict(P=0), -4), (dict(P=3), -4), (dict(M=17, ws_bytes=0), -6), (dict(M=17, ws_bytes=pq.lib().pq_gemm_workspace_bytes(17, 128, 256) - 1), -6),
    (dict(M=17, ws=None), -1), (dict(a=None), -1), (dict(asg=None), -1), (dict(rs=None), -1), (dict(wpk=None), -1), (dict(sz=None), -1), (dict(h=None), -1),
    (dict(a=FAKE + 8), -3), (dict(asg=FAKE + 2), -3), (dict(wpk=FAKE + 8), -3), (dict(sz=FAKE + 2), -3), (dict(h=FAKE + 2), -3), (dict(M=17, ws=FAKE + 8), -3),
    (dict(M=1 << 20, K=1 << 12, ws_bytes=1 << 50), -2), (dict(M=1 << 24, K=128, F=1 << 23, ldh=1 << 23, ws_bytes=1 << 50), -2),
    (dict(M=0), 0), (dict(M=0, a=None, ws=None, ws_bytes=0), 0)])
def test_refusals(kw, code):
    assert _call(**kw) == code


def test_binding_refusals():
    M, K, F = 20, 256, 64
    A, S = torch.zeros(1, M, K, dtype=torch.uint8), torch.zeros(1, M, 2)
    wpk = torch.zeros(pq.lib().pq_packed_weight_bytes(K, 2 * F), dtype=torch.uint8)
    sz = torch.zeros(2, 2 * F, 2, dtype=torch.float16)
    ws = torch.zeros(pq.gemm_workspace_bytes(M, 2 * F, K), dtype=torch.uint8)
    for bad, err in ((dict(A=A[0]), ValueError), (dict(A=A.to(torch.int8)), TypeError), (dict(ASG=S[:, :4]), ValueError), (dict(RS=S.half()), TypeError),
                     (dict(F=72), ValueError), (dict(F=0), ValueError), (dict(F=128), ValueError), (dict(sz=sz[:, :F]), ValueError),
                     (dict(act="relu"), ValueError), (dict(prepared=True), ValueError), (dict(workspace=ws[1:]), ValueError),
                     (dict(out=torch.zeros(M, 32, dtype=torch.float16)), ValueError), (dict(out=torch.zeros(M, F)), TypeError),
                     (dict(dtype=torch.float32), TypeError), (dict(out=torch.zeros(M, F, dtype=torch.float16), dtype=torch.bfloat16), TypeError),
                     (dict(), TypeError)):
        a = dict(A=A, ASG=S, RS=S.clone(), wpk=wpk, sz=sz, F=F)
        a.update(bad)
        with pytest.raises(err):
            pq.gemm_glu(a.pop("A"), a.pop("ASG"), a.pop("RS"), a.pop("wpk"), a.pop("sz"), a.pop("F"), **a)


# ------------------------------------------------------------------------------------------
gpu = pytest.mark.gpu


class Pair:
    def __init__(self, K, F, seed):
        w = synth.weights(synth.Workload("glu", seed, 1, K, 2 * F))
        self.K, self.F, self.G = K, F, K // 128
        self.wpk, self.sz = pq.pack_weights(*(torch.from_numpy(a).cuda() for a in (w.qweight, w.qzeros, w.scales)))
        self.sc = torch.from_numpy(w.scales).cuda().double()
        zp = torch.from_numpy(awq.unpack(w.qzeros).astype(np.float64)).cuda()
        self.c = torch.from_numpy(awq.unpack(w.qweight).astype(np.uint8)).cuda().double()
        self.zsc = (self.sc * (zp - 8)).half().double()


def _codes(P, M, K, seed, one_signed=False):
    """Codes and scales as the prologue leaves them: every group's largest value at 448, a zero group, a zero row."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = torch.randn((P, M, K // 128, 128), generator=g, device="cuda") * torch.exp(torch.randn((P, M, K // 128, 1), generator=g, device="cuda"))
    v = v.abs() if one_signed else v
    v[:, M // 2, K // 256] = 0
    if M > 2:
        v[:, 1] = 0
    asg = v.abs().amax(-1) / 448
    code = torch.where(asg[..., None] > 0, v / asg[..., None], torch.zeros_like(v)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return code.view(torch.uint8).reshape(P, M, K), asg, code.float().sum(-1)


def _check(tag, h, A, S, R, pair, act, rows=None):
    rows = slice(None) if rows is None else rows
    P, M, K = A.shape
    F, G = pair.F, pair.G
    e = torch.finfo(h.dtype).eps / 2
    tiny = 2.0 ** -25 if h.dtype == torch.float16 else 2.0 ** -126
    rep = lambda t: torch.repeat_interleave(t, 128, 0)   # noqa: E731
    out = []
    for s in range(2):
        p, cols = (0 if P == 1 else s), slice(s * F, (s + 1) * F)
        D = A[p, rows].view(torch.float8_e4m3fn).double()
        a = D * torch.repeat_interleave(S[p, rows].double(), 128, -1)
        sc = rep(pair.sc[:, cols])
        v = a @ (sc * (pair.c[:, cols] - 8) - rep(pair.zsc[:, cols]))
        Y = a.abs() @ (sc * pair.c[:, cols])
        Z = (S[p, rows] * R[p, rows]).double().abs() @ (8 * pair.sc[:, cols] + pair.zsc[:, cols]).abs()
        X = a.abs().reshape(a.shape[0], K // 8, 8).amax(-1) @ torch.repeat_interleave(pair.sc[:, cols], 16, 0)
        out.append((v, 7 * 2.0 ** -10 * X + (272 + G) * U24 * Y + (2.0 ** -14 + (3 * G + 16) * U24) * Z))
    (g, Eg), (u, Eu) = out
    a = g * torch.sigmoid(g) if act == "silu" else 0.5 * g * (1 + torch.tanh(np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)))
    ref = a * u
    bound = e * ref.abs() + (1 + e) * (1.13 * Eg * u.abs() + a.abs() * Eu + 1.13 * Eg * Eu + 2.0 ** -14 * ref.abs() + 2.0 ** -118 * u.abs()) + tiny
    got = h[rows].double()
    assert torch.isfinite(got).all(), tag
    ratio = ((got - ref).abs() / bound).max().item()
    rel = ((got - ref).norm() / ref.norm().clamp_min(1e-300)).item()
    print(f"[glu {tag}] worst error/bound {ratio:.3f}, relative {rel:.2e}", flush=True)
    # 2e-3 of the norm for v before its rounding; rounding moves each value by at most e |v|, so the norm by at most
    # e |v| <= e (1 + 2e-3) |ref|. In bf16 (e = 2^-8 = 3.9e-3) that part alone can pass 2e-3 where a few values carry the norm.
    assert ratio <= 1.0 and rel <= 2e-3 + e * (1 + 2e-3), tag


def _run(A, S, R, pair, act="silu", dtype=torch.float16, pad=0, **kw):
    M, F = A.shape[1], pair.F
    buf = torch.full((M + 2, F + pad), 3.0, dtype=dtype, device="cuda")
    assert pq.gemm_glu(A, S, R, pair.wpk, pair.sz, F, act=act, out=buf[:M, :F], **kw).data_ptr() == buf.data_ptr()
    torch.cuda.synchronize()
    assert torch.all(buf[M:] == 3) and torch.all(buf[:, F:] == 3)
    return buf[:M, :F]


@gpu
@pytest.mark.parametrize("M,K,F,P,act,ht,pad", [
    (1, 128, 16, 1, "silu", "f16", 0), (1, 5120, 8704, 1, "silu", "f16", 0), (2, 384, 48, 2, "gelu", "bf16", 2), (8, 5120, 8704, 1, "gelu", "bf16", 0),
    (8, 1152, 8704, 2, "silu", "f16", 8), (9, 640, 8704, 1, "silu", "bf16", 0), (16, 1152, 8704, 2, "gelu", "f16", 2), (16, 256, 13008, 1, "silu", "f16", 0),
    (3, 256, 20496, 1, "gelu", "f16", 0), (5, 128, 20496, 2, "silu", "bf16", 0), (2, 128, 25616, 1, "gelu", "f16", 0), (12, 128, 26000, 2, "silu", "f16", 0), (9, 256, 9216, 1, "silu", "bf16", 2),
    (16, 640, 8704, 2, "gelu", "f16", 0), (1, 256, 16384, 2, "silu", "f16", 0), (1, 17408, 5120, 1, "silu", "f16", 0)])
def test_few_rows(M, K, F, P, act, ht, pad):
    print(f"[glu] M={M} K={K} F={F} P={P} {act} {ht}", flush=True)
    pair = Pair(K, F, 600 + M)
    A, S, R = _codes(P, M, K, M)
    _check(f"M={M} K={K} F={F} P={P}", _run(A, S, R, pair, act, TYPES[ht], pad), A, S, R, pair, act)


@gpu
@pytest.mark.parametrize("M,K,F,P,act,ht,pad", [
    (17, 128, 16, 1, "silu", "f16", 0), (33, 5120, 8704, 1, "silu", "f16", 0), (48, 1280, 8704, 1, "gelu", "bf16", 2), (65, 1152, 8704, 1, "silu", "f16", 0),
    (128, 5120, 8704, 1, "silu", "bf16", 0), (129, 1024, 8704, 1, "silu", "f16", 0), (31, 640, 8704, 2, "gelu", "bf16", 0), (50, 1152, 8704, 2, "silu", "f16", 2),
    (20, 2048, 5120, 1, "silu", "f16", 0), (40, 2048, 2048, 1, "gelu", "bf16", 0), (47, 1152, 1424, 1, "silu", "f16", 2), (33, 1152, 4096, 2, "silu", "bf16", 0),
    (100, 512, 4096, 1, "gelu", "f16", 0), (192, 1024, 2048, 1, "silu", "bf16", 0), (250, 1408, 1600, 2, "gelu", "f16", 0), (30, 640, 7040, 1, "silu", "f16", 0),
    (300, 384, 8704, 1, "silu", "f16", 0), (500, 256, 8208, 1, "gelu", "bf16", 8), (380, 640, 4160, 1, "silu", "f16", 2), (900, 256, 2048, 1, "gelu", "f16", 0),
    (297, 1408, 208, 1, "silu", "f16", 0), (68, 2176, 544, 1, "gelu", "bf16", 2), (844, 768, 32, 1, "silu", "bf16", 0), (33, 1152, 1024, 2, "silu", "f16", 0),
    (18, 1024, 720, 1, "gelu", "f16", 0), (735, 384, 944, 1, "silu", "bf16", 2), (50, 640, 8704, 1, "gelu", "bf16", 0), (1000, 256, 512, 1, "silu", "f16", 0),
    (350, 1024, 352, 1, "gelu", "f16", 0), (19, 5120, 16, 1, "silu", "f16", 0), (4000, 128, 16, 1, "gelu", "bf16", 0), (75, 1664, 128, 2, "gelu", "f16", 2),
    (1300, 256, 4640, 1, "silu", "f16", 0), (1500, 128, 4112, 1, "gelu", "bf16", 2),
    (1200, 384, 8704, 1, "gelu", "bf16", 2), (700, 640, 8704, 2, "silu", "f16", 2), (2000, 256, 512, 1, "silu", "f16", 0), (600, 512, 1024, 1, "gelu", "f16", 0), (17, 256, 48, 2, "gelu", "bf16", 2), (64, 1152, 144, 1, "gelu", "f16", 2), (300, 1024, 1424, 1, "gelu", "bf16", 0),
    (300, 1024, 1424, 2, "silu", "f16", 0), (129, 384, 2064, 2, "silu", "bf16", 8), (513, 640, 4112, 1, "silu", "f16", 0), (257, 256, 8720, 2, "gelu", "f16", 0),
    (1100, 512, 8704, 1, "silu", "bf16", 0), (2048, 256, 8704, 2, "silu", "f16", 0)])
def test_many_rows(M, K, F, P, act, ht, pad):
    print(f"[glu] M={M} K={K} F={F} P={P} {act} {ht}", flush=True)
    pair = Pair(K, F, 620 + M)
    A, S, R = _codes(P, M, K, M)
    _check(f"M={M} K={K} F={F} P={P}", _run(A, S, R, pair, act, TYPES[ht], pad), A, S, R, pair, act)


@gpu
def test_prompt_of_the_headline_layer():
    print("[glu] M=2048 K=5120 F=8704", flush=True)
    pair = Pair(5120, 8704, 640)
    A, S, R = _codes(1, 2048, 5120, 9)
    h = _run(A, S, R, pair)
    _check("M=2048", h, A, S, R, pair, "silu", rows=torch.randperm(2048, device="cuda")[:256].sort().values)


@gpu
@pytest.mark.parametrize("M,K,F,P,act", [(73, 128, 48, 1, "gelu"), (10, 256, 7952, 1, "gelu"), (480, 128, 608, 1, "gelu"), (792, 256, 5632, 2, "silu"), (300, 384, 4464, 1, "silu")])
def test_outlier_channels(M, K, F, P, act):
    """One channel in a hundred 20 times as large: its products' exponent decides what the matrix core keeps of its neighbours'."""
    pair = Pair(K, F, 500 + M)
    g = torch.Generator(device="cuda").manual_seed(M)
    v = torch.randn((P, M, K), generator=g, device="cuda") * torch.exp(0.5 * torch.randn((P, M, 1), generator=g, device="cuda"))
    v[..., torch.randperm(K, generator=g, device="cuda")[:K // 100]] *= 20
    v = v.reshape(P, M, K // 128, 128)
    asg = v.abs().amax(-1) / 448
    code = (v / asg[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    A, S, R = code.view(torch.uint8).reshape(P, M, K), asg, code.float().sum(-1)
    _check(f"outliers M={M}", _run(A, S, R, pair, act), A, S, R, pair, act)


@gpu
@pytest.mark.parametrize("M", [1, 7, 16, 300])
def test_one_signed_rows(M):
    """Codes of one sign: the zero-point term is as large as the products that it cancels."""
    pair = Pair(1024, 528, 650)
    A, S, R = _codes(1, M, 1024, M, one_signed=True)
    _check(f"one-signed M={M}", _run(A, S, R, pair, dtype=torch.bfloat16), A, S, R, pair, "silu")


@gpu
@pytest.mark.parametrize("M", [1, 8, 16, 17, 300, 700, 3000])
def test_two_equal_partitions_are_one(M):
    """The same bits where both forms add the groups in the same order (300 and 700 rows split them differently)."""
    pair = Pair(1152, 2064, 660)
    A, S, R = _codes(1, M, 1152, M)
    both = [t.expand(2, *t.shape[1:]).contiguous() for t in (A, S, R)]
    one, two = _run(A, S, R, pair), _run(*both, pair)
    assert M in (300, 700) or torch.equal(one, two)
    _check(f"equal partitions M={M}", two, *both, pair, "silu")


@gpu
def test_extreme_gates():
    """Gates far to either side (|g| of 100 to 4000): silu and gelu are 0 or g, never NaN."""
    pair = Pair(1024, 256, 670)
    for M in (3, 40):
        A, S, R = _codes(1, M, 1024, M)
        for act in ("silu", "gelu"):
            _check(f"extreme {act} M={M}", _run(A, S * 40, R, pair, act, torch.bfloat16), A, S * 40, R, pair, act)


@gpu
def test_prepared_empty_stream_graph():
    wl = synth.Workload("glu", 680, 300, 1024, 2 * 1040)
    pair = Pair(1024, 1040, 680)
    pl, tl, cl = synth.rotations(wl)
    rec = torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda()
    cs, x = torch.from_numpy(np.stack(cl)).cuda(), torch.from_numpy(synth.activations(wl)).cuda()
    ws = torch.full((pq.gemm_workspace_bytes(300, 2080, 1024),), 0xFF, dtype=torch.uint8, device="cuda")
    A, S, R = pq.rotate_quant_for_gemm(x, rec, cs, ws)
    want = pq.gemm_glu(A, S, R, pair.wpk, pair.sz, 1040)
    got = pq.gemm_glu(A, S, R, pair.wpk, pair.sz, 1040, workspace=ws, prepared=True)
    assert torch.equal(got, want) and want.dtype == torch.float16
    assert pq.gemm_glu(A[:, :0].contiguous(), S[:, :0].contiguous(), R[:, :0].contiguous(), pair.wpk, pair.sz, 1040).shape == (0, 1040)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pq.gemm_glu(A, S, R, pair.wpk, pair.sz, 1040, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    for M in (5, 300):
        a, s, r = (t[:, :M].contiguous() for t in (A, S, R))
        eager = pq.gemm_glu(a, s, r, pair.wpk, pair.sz, 1040)
        out, w = torch.empty_like(eager), torch.empty_like(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pq.gemm_glu(a, s, r, pair.wpk, pair.sz, 1040, out=out, workspace=w)
        for k in range(3):
            out.zero_()
            g.replay()
            again = pq.gemm_glu(a, s, r, pair.wpk, pair.sz, 1040)
            torch.cuda.synchronize()
            assert torch.equal(out, eager) and torch.equal(again, eager), (M, k)
