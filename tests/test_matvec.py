"""pq_matvec: refusals (CPU) and parity with the formula in 64 bits (GPU).

    y = sum_k x W,  W = sc (c - 8) - zsc,  zsc = fl16(sc (zp - 8))

Tolerance. The kernel adds up x c on the matrix core (exact 16-bit products, 128 terms in binary32 in any order,
doubled for a truncating adder: 2 * 128 u), the sums of x likewise, then per group two products, two sums and the
factor 8 sc + zsc (exact), then 8 partial sums:

    |y - y_ref| <= e |y_ref| + (1 + e) (2*128 + 3G + 16) u sum_g (sc sum|x| c + |8 sc + zsc| sum|x|) + tiny

with u = 2^-24, e = eps/2 of y's type, tiny half its smallest subnormal (bf16: the smallest normal)."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
from oracle import awq

U = 2.0 ** -24
FAKE = 0x100000000
NB = pq.NO_BOUNDARY
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _call(**kw):
    a = dict(x=FAKE, ldx=256, xt=0, M=4, K=256, P=1, wpk=FAKE, sz=FAKE, N=128, pb1=NB, pb2=NB, y=FAKE, ldy=128, yt=0, s=None)
    a.update(kw)
    return pq.lib().pq_matvec(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -2), (dict(M=17), -2), (dict(K=0), -2), (dict(K=100), -2), (dict(N=0), -2), (dict(N=120), -2), (dict(xt=2), -2), (dict(yt=2), -2),
    (dict(ldx=248), -2), (dict(ldx=260), -2), (dict(ldx=(1 << 26) + 8), -2), (dict(ldy=126), -2), (dict(ldy=129), -2),
    (dict(P=0), -4), (dict(P=2), -4), (dict(P=1, pb1=128, N=256, ldy=256), -4), (dict(P=2, pb1=64), -4), (dict(P=4), -4),
    (dict(x=None), -1), (dict(wpk=None), -1), (dict(sz=None), -1), (dict(y=None), -1),
    (dict(x=FAKE + 8), -3), (dict(wpk=FAKE + 4), -3), (dict(sz=FAKE + 2), -3), (dict(y=FAKE + 2), -3),
    (dict(M=0), 0), (dict(M=0, x=None, y=None), 0)])
def test_refusals(kw, code):
    assert _call(**kw) == code


def test_binding_refusals():
    K, N = 256, 128
    x = torch.zeros(4, K, dtype=torch.float16)
    wpk = torch.zeros(pq.lib().pq_packed_weight_bytes(K, N), dtype=torch.uint8)
    sz = torch.zeros(K // 128, N, 2, dtype=torch.float16)
    for bad, err in ((dict(x=x.float()), TypeError), (dict(x=torch.zeros(17, K, dtype=torch.float16)), ValueError), (dict(x=x[0]), ValueError),
                     (dict(x=x[:, :100]), ValueError), (dict(N=120), ValueError), (dict(wpk=wpk[1:]), ValueError), (dict(sz=sz[:1]), ValueError),
                     (dict(sz=sz.float()), TypeError), (dict(out=torch.zeros(3, N, dtype=torch.float16)), ValueError),
                     (dict(out=torch.zeros(4, 64, dtype=torch.float16)), ValueError), (dict(out=torch.zeros(4, N)), TypeError),
                     (dict(dtype=torch.float32), TypeError), (dict(out=torch.zeros(4, N, dtype=torch.float16), dtype=torch.bfloat16), TypeError),
                     (dict(), TypeError)):
        a = dict(x=x, wpk=wpk, sz=sz, N=N)
        a.update(bad)
        with pytest.raises(err):
            pq.matvec(a.pop("x"), a.pop("wpk"), a.pop("sz"), a.pop("N"), **a)


# ------------------------------------------------------------------------------------------
gpu = pytest.mark.gpu


class Layer:
    def __init__(self, K, N, seed):
        w = synth.weights(synth.Workload("mv", seed, 1, K, N))
        self.K, self.N, self.G = K, N, K // 128
        self.wpk, self.sz = pq.pack_weights(*(torch.from_numpy(a).cuda() for a in (w.qweight, w.qzeros, w.scales)))
        sc = torch.from_numpy(w.scales).cuda().double()
        zp = torch.from_numpy(awq.unpack(w.qzeros).astype(np.float64)).cuda()
        c = torch.from_numpy(awq.unpack(w.qweight).astype(np.uint8)).cuda().double()
        zsc = (sc * (zp - 8)).half().double()
        rep = lambda t: torch.repeat_interleave(t, 128, 0)   # noqa: E731
        self.W = rep(sc) * (c - 8) - rep(zsc)
        self.mag = rep(sc) * c + rep((8 * sc + zsc).abs())


def _check(tag, y, x, layer, cuts):
    """x [P, M, K]; cuts the partitions' column ranges."""
    e = torch.finfo(y.dtype).eps / 2
    tiny = 2.0 ** -25 if y.dtype == torch.float16 else 2.0 ** -126
    worst = 0.0
    for p, (a, b) in enumerate(cuts):
        ref = x[p].double() @ layer.W[:, a:b]
        bound = e * ref.abs() + (1 + e) * (256 + 3 * layer.G + 16) * U * (x[p].double().abs() @ layer.mag[:, a:b]) + tiny
        worst = max(worst, ((y[:, a:b].double() - ref).abs() / bound).max().item())
    print(f"[matvec {tag}] worst error/bound {worst:.3f}", flush=True)
    assert worst <= 1.0, tag


def _x(P, M, K, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((P, M, K), generator=g, device="cuda") * torch.exp(torch.randn((P, M, 1), generator=g, device="cuda"))
    x[..., torch.randperm(K, generator=g, device="cuda")[:max(1, K // 100)]] *= 20
    return x.to(dtype)


def _run(x, layer, pb1=NB, pb2=NB, dtype=None, pad=0):
    M, N = x.shape[-2], layer.N
    buf = torch.full((M + 2, N + pad), 3.0, dtype=dtype or x.dtype, device="cuda")
    y = buf[:M, :N]
    assert pq.matvec(x, layer.wpk, layer.sz, N, pb1, pb2, out=y).data_ptr() == y.data_ptr()
    torch.cuda.synchronize()
    assert torch.all(buf[M:] == 3) and torch.all(buf[:, N:] == 3)
    return y


@gpu
@pytest.mark.parametrize("K,N", [(128, 16), (256, 128), (1152, 48), (640, 8208), (5120, 1040)])
def test_every_row_count(K, N):
    layer = Layer(K, N, 500 + N)
    for M in range(1, 17):
        for xt, yt in (("f16", "bf16"), ("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16"))[M % 2::2]:
            print(f"[matvec] M={M} K={K} N={N} {xt} -> {yt}", flush=True)
            x = _x(1, M, K, TYPES[xt], M)
            _check(f"M={M} {xt} {yt}", _run(x, layer, dtype=TYPES[yt], pad=2 * (M % 3)), x, layer, [(0, N)])


@gpu
@pytest.mark.parametrize("M,K,N,xt", [(1, 5120, 17408, "f16"), (8, 5120, 17408, "bf16"), (16, 5120, 17408, "f16"), (1, 17408, 5120, "bf16"),
                                      (16, 17408, 5120, "f16"), (3, 256, 40976, "f16"), (16, 256, 40976, "bf16"), (16, 128, 19472, "f16"),
                                      (1, 256, 33792, "bf16"), (1, 128, 34000, "f16"), (4, 384, 29696, "f16"), (2, 128, 30000, "bf16"), (8, 256, 25600, "bf16"),
                                      (5, 640, 20496, "f16"), (16, 256, 29696, "f16"), (12, 1152, 24576, "bf16"), (9, 128, 18432, "f16"), (1, 128, 70000, "f16")])
def test_layer_sizes(M, K, N, xt):
    print(f"[matvec] M={M} K={K} N={N} {xt}", flush=True)
    layer = Layer(K, N, 520 + M)
    x = _x(1, M, K, TYPES[xt], M)
    _check(f"M={M} K={K} N={N}", _run(x, layer), x, layer, [(0, N)])


@gpu
@pytest.mark.parametrize("M,K,cuts,xt", [(4, 5120, (6144, 1024, 1024), "bf16"), (1, 384, (128, 48), "f16"), (16, 640, (256, 128, 144), "bf16"),
                                         (7, 1024, (1280, 128), "f16"), (6, 256, (3584, 15616, 3136), "bf16"), (16, 256, (8192, 8192, 1040), "f16"),
                                         (1, 128, (16384, 384, 16624), "bf16"), (12, 384, (128, 20352, 16), "bf16")])
def test_partitions(M, K, cuts, xt):
    N, ends = sum(cuts), np.cumsum(cuts).tolist()
    layer = Layer(K, N, 540 + M)
    x = _x(len(cuts), M, K, TYPES[xt], M)
    pb = (ends[:-1] + [NB] * 2)[:2]
    print(f"[matvec] M={M} K={K} {cuts} {xt}", flush=True)
    _check(f"{cuts}", _run(x, layer, *pb), x, layer, list(zip([0] + ends[:-1], ends)))
    same = x[:1].expand(len(cuts), M, K).contiguous()   # the same rows in every partition
    _check("equal", _run(same, layer, *pb), same, layer, list(zip([0] + ends[:-1], ends)))


@gpu
def test_codes_zeros_subnormals_and_strides():
    """Every code and zero point in every column, unit rows (one weight a product), f16 subnormals, strided rows."""
    K, N = 256, 64
    codes = (np.arange(K)[:, None] + np.arange(N)[None]) % 16
    zp = (np.arange(2)[:, None] * 8 + np.arange(N)[None]) % 16
    sc = np.full((2, N), 0.5, np.float16)
    wpk, sz = pq.pack_weights(*(torch.from_numpy(a).cuda() for a in (synth.awq_pack(codes.astype(np.uint8)), synth.awq_pack(zp.astype(np.uint8)), sc)))
    W = 0.5 * (codes - np.repeat(zp, 128, axis=0))             # exact in every type
    for dtype in (torch.float16, torch.bfloat16):
        for k0 in range(0, K, 16):
            x = torch.zeros((16, K + 8), dtype=dtype, device="cuda")[:, :K]
            x[torch.arange(16), torch.arange(k0, k0 + 16)] = 1
            y = pq.matvec(x, wpk, sz, N)
            assert np.array_equal(y.double().cpu().numpy(), W[k0:k0 + 16]), (dtype, k0)
        assert not pq.matvec(torch.zeros((1, K), dtype=dtype, device="cuda"), wpk, sz, N).any()
    x = torch.zeros((5, K), dtype=torch.float16, device="cuda")
    x[torch.arange(5), torch.tensor([0, 77, 130, 200, 255])] = 2.0 ** -24       # the smallest subnormal
    y = pq.matvec(x, wpk, sz, N, dtype=torch.bfloat16)
    assert np.array_equal(y.double().cpu().numpy(), 2.0 ** -24 * W[[0, 77, 130, 200, 255]])


@gpu
def test_non_finite_rows_empty_stream_graph():
    layer = Layer(1024, 512, 560)
    x = _x(1, 6, 1024, torch.float16, 1)[0].contiguous()
    want = pq.matvec(x, layer.wpk, layer.sz, 512)
    assert pq.matvec(x[:0], layer.wpk, layer.sz, 512).shape == (0, 512)
    bad = x.clone()
    bad[2, 700], bad[4, 3] = float("nan"), float("inf")
    y = pq.matvec(bad, layer.wpk, layer.sz, 512)
    assert torch.equal(y[[0, 1, 3, 5]], want[[0, 1, 3, 5]]) and torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pq.matvec(x, layer.wpk, layer.sz, 512, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.matvec(x, layer.wpk, layer.sz, 512, out=out)
    for r in range(3):
        out.zero_()
        g.replay()
        eager = pq.matvec(x, layer.wpk, layer.sz, 512)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(out, want), r
