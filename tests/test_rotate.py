"""pq_rotate: refusals (CPU), bit parity with the prologue's binary32 arithmetic and a bound against the
rotation in 64 bits (GPU).

Against 64 bits, u = 2^-24: every layer writes each value as a sum of two products, three roundings of terms no larger than
the pair's norm, so it adds at most 3 sqrt(2) u times the group's norm, which a layer keeps up to the f16 rounding of
cos and sin (a factor below 1 + 2^-10); over 8 layers at most 36 u ||x cs||_group:

    |y - y_ref| <= e |y_ref| + 1.01 * 36 u ||(x cs)_group||_2 + tiny,   e = eps/2 of y's type"""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
from oracle import prologue as opro
from oracle import records as orec

U = 2.0 ** -24
FAKE = 0x100000000


def _call(**kw):
    a = dict(x=FAKE, ldx=256, xt=0, M=4, K=256, P=1, rec=FAKE, cs=FAKE, y=FAKE + (1 << 20), s=None)
    a.update(kw)
    return pq.lib().pq_rotate(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(M=-1), -2), (dict(K=0), -2), (dict(K=100), -2), (dict(xt=2), -2), (dict(xt=-1), -2), (dict(P=0), -4), (dict(P=4), -4),
    (dict(ldx=254), -2), (dict(ldx=257), -2), (dict(ldx=(1 << 26) + 8), -2), (dict(x=None), -1), (dict(rec=None), -1), (dict(cs=None), -1), (dict(y=None), -1),
    (dict(x=FAKE + 2), -3), (dict(rec=FAKE + 4), -3), (dict(cs=FAKE + 2), -3), (dict(y=FAKE + (1 << 20) + 8), -3),
    (dict(y=FAKE), -2), (dict(y=FAKE + 1024), -2), (dict(x=FAKE + (1 << 20) + 1536, P=1), -2), (dict(x=FAKE + (1 << 20) + 4096, P=3), -2),
    (dict(M=0), 0), (dict(M=0, x=None, y=None), 0)])
def test_refusals(kw, code):
    assert _call(**kw) == code


def test_binding_refusals():
    x, rec, cs = torch.zeros(4, 256, dtype=torch.float16), torch.zeros(1, 8, 128, 8, dtype=torch.uint8), torch.ones(1, 256, dtype=torch.float16)
    for bad, err in ((dict(x=x.float()), TypeError), (dict(x=x[0]), ValueError), (dict(x=x[:, :100]), ValueError),
                     (dict(rec=rec[:, :, :64]), ValueError), (dict(cs=cs[:, :128]), ValueError), (dict(cs=cs.bfloat16()), TypeError),
                     (dict(out=torch.zeros(1, 4, 128, dtype=torch.float16)), ValueError),
                     (dict(out=torch.zeros(1, 4, 256, dtype=torch.bfloat16)), TypeError), (dict(), TypeError)):
        a = dict(x=x, rec=rec, cs=cs)
        a.update(bad)
        with pytest.raises(err):
            pq.rotate(a.pop("x"), a.pop("rec"), a.pop("cs"), **a)


# ------------------------------------------------------------------------------------------
gpu = pytest.mark.gpu


def _rotate32(x, rec, cs):
    """The prologue's steps 1-2 on float32 values of any 16-bit type (numpy rounds every product and sum)."""
    v = x.astype(np.float32) * cs.astype(np.float32)
    base = (np.arange(v.shape[1] // 2) // 64) * 128
    for r in range(8):
        i, j, c, s = rec["i"][r] + base, rec["j"][r] + base, rec["cos"][r], rec["sin"][r]
        a, b = v[:, i].copy(), v[:, j].copy()
        v[:, i], v[:, j] = (c * a) + (s * b), (c * b) - (s * a)
    return v


def _rotate64(x, rec, cs):
    v = x.astype(np.float64) * cs.astype(np.float64)
    norm = np.repeat(np.linalg.norm(v.reshape(len(v), -1, 128), axis=-1), 128, axis=-1)
    base = (np.arange(v.shape[1] // 2) // 64) * 128
    for r in range(8):
        i, j, c, s = rec["i"][r] + base, rec["j"][r] + base, rec["cos"][r].astype(np.float64), rec["sin"][r].astype(np.float64)
        a, b = v[:, i].copy(), v[:, j].copy()
        v[:, i], v[:, j] = c * a + s * b, c * b - s * a
    return v, norm


@gpu
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M,K,splits,pad", [(1, 128, (), 0), (1, 5120, (), 0), (3, 384, (64, 64), 2), (9, 640, (64, 32, 32), 0), (37, 1152, (), 8),
                                            (130, 256, (64, 64), 6), (257, 5120, (), 0), (8, 17408, (), 0)])
def test_parity(dtype, M, K, splits, pad):
    print(f"[rotate] {dtype} M={M} K={K} P={max(1, len(splits))} pad={pad}", flush=True)
    wl = synth.Workload("rot", 300 + M, M, K, 128, splits=splits, outliers=True)
    x32 = torch.from_numpy(synth.activations(wl).astype(np.float32))
    pl, tl, cl = synth.rotations(wl)
    rec = torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda()
    buf = torch.zeros((M, K + pad), dtype=dtype, device="cuda")
    x = buf[:, :K]
    x.copy_(x32.cuda())
    whole = torch.full((len(pl) * M * K + 512,), 3.0, dtype=dtype, device="cuda")
    y = whole[:len(pl) * M * K].view(len(pl), M, K)
    assert pq.rotate(x, rec, torch.from_numpy(np.stack(cl)).cuda(), out=y) is y
    torch.cuda.synchronize()
    assert torch.all(whole[y.numel():] == 3)
    xs = x.float().cpu().numpy()
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -126
    for p in range(len(pl)):
        ref = orec.build(pl[p], tl[p])
        want = torch.from_numpy(_rotate32(xs, ref, cl[p])).to(dtype)
        assert torch.equal(y[p].cpu(), want)
        if dtype == torch.float16:
            assert np.array_equal(_rotate32(xs, ref, cl[p]), opro.rotate_f32(x.cpu().numpy(), ref, cl[p]))
        y64, norm = _rotate64(xs, ref, cl[p])
        bound = torch.finfo(dtype).eps / 2 * np.abs(y64) + 1.01 * 36 * U * norm + tiny
        ratio = (np.abs(y[p].double().cpu().numpy() - y64) / bound).max()
        print(f"[rotate] partition {p}: bits equal, worst error/bound against 64 bits {ratio:.3f}", flush=True)
        assert ratio <= 1.0


@gpu
def test_rows_apart_empty_stream_graph():
    wl = synth.Workload("rot", 400, 21, 512, 128, splits=(64, 64))
    pl, tl, cl = synth.rotations(wl)
    rec = torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda()
    cs = torch.from_numpy(np.stack(cl)).cuda()
    x = torch.from_numpy(synth.activations(wl)).cuda()
    assert pq.rotate(x[:0], rec, cs).shape == (2, 0, 512)
    want = pq.rotate(x, rec, cs)
    bad = x.clone()
    bad[4, 200] = float("nan")
    got = pq.rotate(bad, rec, cs)
    keep = torch.ones_like(got, dtype=torch.bool)
    keep[:, 4, 128:256] = False                      # a NaN stays in its row's group
    assert torch.equal(got[keep], want[keep])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pq.rotate(x, rec, cs, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    y = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.rotate(x, rec, cs, out=y)
    for r in range(3):
        y.zero_()
        g.replay()
        eager = pq.rotate(x, rec, cs)
        torch.cuda.synchronize()
        assert torch.equal(y, eager) and torch.equal(y, want), r
