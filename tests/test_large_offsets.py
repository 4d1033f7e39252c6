"""rotate, matvec, gemm_glu and block_norms on tensors whose element offsets pass 32 bits: the last rows and columns against
the formulas of the operators' own test files (GPU, up to about 45 GB of device memory)."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
import test_block_norms as tn
import test_gemm_glu as tg
import test_matvec as tm
import test_rotate as tr
from oracle import awq
from oracle import records as orec

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    yield
    torch.cuda.empty_cache()


class Columns:
    """The columns [a, b) of a large layer, for the checks of tm (Layer) and tg (Pair)."""

    def __init__(self, qweight, qzeros, scales, ranges):
        pick = lambda t, w: torch.cat([t[:, a // w:b // w] for a, b in ranges], 1).cpu().numpy()   # noqa: E731
        self.sc = torch.from_numpy(pick(scales, 1)).cuda().double()
        zp = torch.from_numpy(awq.unpack(pick(qzeros, 8)).astype(np.float64)).cuda()
        self.c = torch.from_numpy(awq.unpack(pick(qweight, 8)).astype(np.uint8)).cuda().double()
        self.zsc = (self.sc * (zp - 8)).half().double()
        self.G = self.sc.shape[0]
        rep = lambda t: torch.repeat_interleave(t, 128, 0)   # noqa: E731
        self.W = rep(self.sc) * (self.c - 8) - rep(self.zsc)
        self.mag = rep(self.sc) * self.c + rep((8 * self.sc + self.zsc).abs())
        self.F = self.sc.shape[1] // 2


def test_weights_past_4_gib():
    K, N = 16384, 786432                      # 6.4 GB of codes
    g = torch.Generator(device="cuda").manual_seed(1)
    word = lambda r: torch.randint(-2 ** 31, 2 ** 31 - 1, (r, N // 8), generator=g, device="cuda", dtype=torch.int32)   # noqa: E731
    qw, qz = word(K), word(K // 128)
    sc = (0.002 + 0.018 * torch.rand((K // 128, N), generator=g, device="cuda")).half()
    print("[large] packing 6.4 GB", flush=True)
    wpk, sz = pq.pack_weights(qw, qz, sc)
    F = N // 2
    last = Columns(qw, qz, sc, [(N - 64, N)])
    pair = Columns(qw, qz, sc, [(F - 48, F), (N - 48, N)])
    del qw, qz
    for M in (1, 16):
        print(f"[large] matvec M={M}", flush=True)
        x = tm._x(1, M, K, torch.float16, M)
        y = pq.matvec(x, wpk, sz, N, dtype=torch.bfloat16)
        tm._check(f"last columns M={M}", y[:, -64:], x, last, [(0, 64)])
    for M in (1, 16, 40, 300):
        print(f"[large] gemm_glu M={M}", flush=True)
        A, S, R = tg._codes(1, M, K, M)
        h = pq.gemm_glu(A, S, R, wpk, sz, F, dtype=torch.bfloat16)
        tg._check(f"last columns M={M}", h[:, -48:], A, S, R, pair, "silu")


def test_outputs_past_32_bits():
    M, K, F = 600_003, 128, 8192              # 4.9e9 outputs
    pair = tg.Pair(K, F, 801)
    A, S, R = tg._codes(1, 4096, K, 3)
    A, S, R = (t.repeat(1, 147, *([1] * (t.dim() - 2)))[:, :M].contiguous() for t in (A, S, R))
    print("[large] gemm_glu rows", flush=True)
    h = pq.gemm_glu(A, S, R, pair.wpk, pair.sz, F)
    rows = torch.tensor([0, 524287, 524288, M - 300, M - 2, M - 1], device="cuda")
    tg._check("last rows", h, A, S, R, pair, "silu", rows=rows)


def test_rows_past_32_bits():
    M, K = 600_001, 8192                      # 4.9e9 elements
    print("[large] block_norms", flush=True)
    x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    res = torch.empty((M, K), dtype=torch.float16, device="cuda")
    rows = torch.tensor([0, 262144, 524288, M - 2, M - 1], device="cuda")
    xs, rs, wp, gt, wn = tn._inputs(5, K, torch.bfloat16, torch.float16, torch.float16, "channel", 4)
    x.fill_(1)
    res.fill_(1)
    x[rows], res[rows] = xs, rs
    h, hs = pq.block_norms(x, res, wp, gt, wn, residual_out=res)
    tn._check("last rows", (h[rows], hs[rows]), tn._reference(xs, rs, wp, gt, 1e-6, 1.0, 1.0, "none", False), wn, 1e-6, False)
    del h, hs, res
    print("[large] rotate", flush=True)
    wl = synth.Workload("rot", 810, 5, K, 128, splits=(64, 64))
    pl, tl, cl = synth.rotations(wl)
    rec = torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda()
    y = pq.rotate(x, rec, torch.from_numpy(np.stack(cl)).cuda())
    for p in range(2):
        want = torch.from_numpy(tr._rotate32(xs.float().cpu().numpy(), orec.build(pl[p], tl[p]), cl[p])).to(torch.bfloat16)
        assert torch.equal(y[p][rows].cpu(), want)
