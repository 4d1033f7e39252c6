"""pq_gemm_glu from the rows on at which it reads its workspace: the 128 x 128 tiles and the 256 x 256 tiles of one rotation and the
tiles of two, which the row blocks of smaller calls never reach (GPU). The bounds are those of test_gemm_glu, which derives them."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
import test_gemm_glu as tg

pytestmark = pytest.mark.gpu

# M, K, F, P: 128 x 128 tiles (less than a round of large ones; two groups), 256 x 256 tiles, the tiles of two rotations (whole and halved)
TILES = [(800, 1152, 2064, 1), (1300, 256, 4640, 1), (1100, 512, 8704, 1), (700, 640, 8704, 2), (2048, 384, 8704, 2)]


def _rotated(M, K, F, P, seed):
    """The prologue of the pair's rotations: x, records, channel scales."""
    wl = synth.Workload("tiles", seed, M, K, P * 128, splits=(128,) * P if P > 1 else ())
    pl, tl, cl = synth.rotations(wl)
    rec = torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda()
    return torch.from_numpy(synth.activations(wl)).cuda(), rec, torch.from_numpy(np.stack(cl)).cuda()


def _workspace(M, F, K):
    return torch.full((pq.gemm_workspace_bytes(M, 2 * F, K),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("M,K,F,P", TILES)
def test_prepared(M, K, F, P):
    """rotate_quant_for_gemm fills the workspace that the call reads instead of ASG and RS: the same bits as without it."""
    print(f"[glu tiles] prepared M={M} K={K} F={F} P={P}", flush=True)
    pair = tg.Pair(K, F, 800 + P)
    x, rec, cs = _rotated(M, K, F, P, 810 + M % 89)
    ws = _workspace(M, F, K)
    A, S, R = pq.rotate_quant_for_gemm(x, rec, cs, ws)
    assert A.shape == (P, M, K)
    want = tg._run(A, S, R, pair)
    tg._check(f"unprepared M={M} P={P}", want, A, S, R, pair, "silu", rows=torch.arange(0, M, 5, device="cuda"))
    assert torch.equal(tg._run(A, S, R, pair, workspace=ws, prepared=True), want)
    # it is the workspace that is read: other ASG and RS change nothing, another workspace everything
    assert torch.equal(tg._run(A, torch.zeros_like(S), torch.zeros_like(R), pair, workspace=ws, prepared=True), want)
    assert torch.isnan(tg._run(A, S, R, pair, workspace=_workspace(M, F, K), prepared=True)).all()
    # on another stream, the prologue and the call on that stream's own order
    ws.fill_(0xFF)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    codes = pq.rotate_quant_for_gemm(x, rec, cs, ws, stream=side)
    prepared = pq.gemm_glu(*codes, pair.wpk, pair.sz, F, workspace=ws, prepared=True, stream=side)
    own = pq.gemm_glu(*codes, pair.wpk, pair.sz, F, stream=side)
    side.synchronize()
    assert torch.equal(prepared, want) and torch.equal(own, want)


@pytest.mark.parametrize("M,K,F,P", TILES)
def test_captured(M, K, F, P):
    """Both forms captured, the plain one with a given workspace and with one of its own; replayed on new rows between eager calls."""
    print(f"[glu tiles] captured M={M} K={K} F={F} P={P}", flush=True)
    pair = tg.Pair(K, F, 820 + P)
    x, rec, cs = _rotated(M, K, F, P, 830 + M % 89)
    ws, ws2 = _workspace(M, F, K), _workspace(M, F, K)
    A, S, R = pq.rotate_quant_for_gemm(x, rec, cs, ws)
    call = lambda **kw: pq.gemm_glu(A, S, R, pair.wpk, pair.sz, F, **kw)   # noqa: E731
    outs = [torch.empty((M, F), dtype=torch.float16, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pq.rotate_quant_for_gemm(x, rec, cs, ws, out=(A, S, R))
        call(out=outs[0], workspace=ws, prepared=True)
        call(out=outs[1], workspace=ws2)
        outs.append(call())
    rows = synth.activations(synth.Workload("tiles", 840, M, K, 128))
    for r in range(3):
        x.copy_(torch.from_numpy(np.roll(rows, r, axis=0)))
        for t in outs:
            t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        codes = pq.rotate_quant(x, rec, cs)
        eager = pq.gemm_glu(*codes, pair.wpk, pair.sz, F)
        torch.cuda.synchronize()
        assert all(torch.equal(t, eager) for t in got), r


def test_two_graphs_share_a_workspace():
    """Replayed one after the other on one stream, each writes the workspace before it reads it."""
    shapes = [(800, 1152, 2064, 1), (700, 640, 8704, 2)]
    ws = torch.empty(max(pq.gemm_workspace_bytes(M, 2 * F, K) for M, K, F, _ in shapes), dtype=torch.uint8, device="cuda")
    graphs = []
    for M, K, F, P in shapes:
        pair, codes = tg.Pair(K, F, 850 + P), tg._codes(P, M, K, M)
        want = pq.gemm_glu(*codes, pair.wpk, pair.sz, F)
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pq.gemm_glu(*codes, pair.wpk, pair.sz, F, out=out, workspace=ws)
        graphs.append((g, out, want, pair, codes))
    for r in range(3):
        for _, out, *_ in graphs:
            out.fill_(7)
        for g, *_ in graphs[::-1] if r == 1 else graphs:
            g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out, want) for _, out, want, *_ in graphs), r


@pytest.mark.parametrize("ht", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,F,P", [(1, 1024, 528, 1), (7, 1024, 528, 1), (16, 1024, 528, 1), (300, 1024, 528, 1)] + TILES)
def test_one_signed_rows(M, K, F, P, ht):
    """Codes of one sign, where the zero-point term (on the tiles a product of bf16 pieces) is as large as the products that it
    cancels; the group scales an eighth, which keeps |h| (up to 1.6e5 without) in f16."""
    print(f"[glu tiles] one-signed M={M} K={K} F={F} P={P} {ht}", flush=True)
    pair = tg.Pair(K, F, 860)
    A, S, R = tg._codes(P, M, K, M, one_signed=True)
    S = S / 8
    _some(f"one-signed M={M} P={P} {ht}", tg._run(A, S, R, pair, dtype=tg.TYPES[ht]), A, S, R, pair, "silu")


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,F,P", TILES)
def test_outlier_channels(M, K, F, P, act):
    """One channel in a hundred 20 times as large."""
    print(f"[glu tiles] outliers M={M} K={K} F={F} P={P} {act}", flush=True)
    pair = tg.Pair(K, F, 870)
    g = torch.Generator(device="cuda").manual_seed(M)
    v = torch.randn((P, M, K), generator=g, device="cuda") * torch.exp(0.5 * torch.randn((P, M, 1), generator=g, device="cuda"))
    v[..., torch.randperm(K, generator=g, device="cuda")[:K // 100]] *= 20
    v = v.reshape(P, M, K // 128, 128)
    S = v.abs().amax(-1) / 448
    code = (v / S[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    A, R = code.view(torch.uint8).reshape(P, M, K), code.float().sum(-1)
    _some(f"outliers M={M} P={P} {act}", tg._run(A, S, R, pair, act), A, S, R, pair, act)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("M,K,F,P", TILES)
def test_extreme_gates(M, K, F, P, act):
    """Gates of hundreds to thousands to either side."""
    print(f"[glu tiles] extreme M={M} K={K} F={F} P={P} {act}", flush=True)
    pair = tg.Pair(K, F, 880)
    A, S, R = tg._codes(P, M, K, M)
    _some(f"extreme M={M} P={P} {act}", tg._run(A, S * 40, R, pair, act, torch.bfloat16), A, S * 40, R, pair, act)


def _some(tag, h, A, S, R, pair, act):
    """The check on about 260 rows, the first and the last among them (every row of fewer)."""
    M = A.shape[1]
    rows = torch.unique(torch.linspace(0, M - 1, min(M, 260), device="cuda").round().long())
    assert torch.isfinite(h).all(), tag
    tg._check(tag, h, A, S, R, pair, act, rows=rows)
