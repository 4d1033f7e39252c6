"""The operators around the packed linear layer together, as a served block uses them (GPU).

A block's feed-forward half with sandwich norms and a gated residual:

    hs = block_norms(attention output, stream)      post-norm, residual, pre-norm
    A = rotate_quant(hs);  h = gemm_glu(A)          gate | up
    B = rotate_quant(h);   y = gemm(B)              down
    stream', hs' = block_norms(y, stream)           post-norm with the block's gate, residual scale, next pre-norm

and the one-token form with 16-bit activations: block_norms -> rotate -> matvec. Every step is checked against its
formula in 64 bits on what the step before really wrote, so the tolerances are those of the single operators (their
test files derive them); the 16-bit chain is also checked end to end."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
import test_block_norms as tn
import test_gemm_glu as tg
import test_matvec as tm

pytestmark = pytest.mark.gpu

K, F = 1024, 1424


class Block:
    def __init__(self, seed=700, F=F):
        self.F = F
        self.pair, self.down = tg.Pair(K, F, seed), tm.Layer(F // 128 * 128, K, seed + 1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [(1 + 0.2 * torch.randn(K, generator=g, device="cuda")).half() for _ in range(4)]
        self.gate = torch.randn(K, generator=g, device="cuda").bfloat16()
        self.rot = {}
        for name, width in (("in", K), ("mid", F // 128 * 128)):
            pl, tl, cl = synth.rotations(synth.Workload("ffn", seed, 1, width, 128))
            self.rot[name] = (torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda(), torch.from_numpy(np.stack(cl)).cuda())

    def inputs(self, M, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        return (torch.randn((M, K), generator=g, device="cuda").bfloat16(), (3 * torch.randn((M, K), generator=g, device="cuda")).half())

    def forward(self, att, stream, keep):
        """Every intermediate goes into ``keep`` (the last call's buffers are reused where they are there already)."""
        M, rq = att.shape[0], self.rot
        width = self.F // 128 * 128
        keep["stream1"], keep["hs"] = pq.block_norms(att, stream, self.w[0], None, self.w[1], gemma=False,
                                                     residual_out=keep.get("stream1"), out=keep.get("hs"))
        n = max(1, pq.gemm_workspace_bytes(M, 2 * self.F, K))
        ws = keep.setdefault("ws", torch.empty(n, dtype=torch.uint8, device="cuda"))
        keep["A"] = pq.rotate_quant_for_gemm(keep["hs"], *rq["in"], ws, out=keep.get("A"))
        keep["h"] = pq.gemm_glu(*keep["A"], self.pair.wpk, self.pair.sz, self.F, out=keep.get("h"), workspace=ws, prepared=True)
        keep["B"] = pq.rotate_quant(keep["h"][:, :width], *rq["mid"], out=keep.get("B"))
        m = pq.gemm_workspace_bytes(M, K, width)
        ws2 = keep.setdefault("ws2", torch.empty(max(1, m), dtype=torch.uint8, device="cuda"))
        keep["y"] = pq.gemm(*keep["B"], self.down.wpk, self.down.sz, K, out=keep.get("y"), workspace=ws2)
        keep["stream2"], keep["hs2"] = pq.block_norms(keep["y"], keep["stream1"], self.w[2], self.gate, self.w[3], scale=0.5, gate_act="sigmoid",
                                                      residual_out=keep.get("stream2"), out=keep.get("hs2"))
        return keep["stream2"], keep["hs2"]


@pytest.mark.parametrize("M", [1, 5, 16, 40, 300])
def test_feed_forward_half(M):
    b, k = Block(), {}
    att, stream = b.inputs(M, M)
    b.forward(att, stream, k)
    torch.cuda.synchronize()
    tn._check(f"into M={M}", (k["stream1"], k["hs"]), tn._reference(att, stream, b.w[0], None, 1e-6, 1.0, 1.0, "none", False), b.w[1], 1e-6, False)
    tg._check(f"block M={M}", k["h"], *k["A"], b.pair, "silu")
    # the down projection on its own codes: the products of the decoded rows, bf16 out
    A, S, R = k["B"]
    a = A[0].view(torch.float8_e4m3fn).double() * torch.repeat_interleave(S[0].double(), 128, -1)
    ref = a @ b.down.W
    assert ((k["y"].double() - ref).norm() / ref.norm()).item() <= 2e-3
    tn._check(f"out of M={M}", (k["stream2"], k["hs2"]), tn._reference(k["y"], k["stream1"], b.w[2], b.gate, 1e-6, 0.5, 1.0, "sigmoid", False),
              b.w[3], 1e-6, False)


@pytest.mark.parametrize("M,dtype", [(1, torch.float16), (3, torch.bfloat16), (16, torch.float16)])
def test_sixteen_bit_form(M, dtype):
    """block_norms -> rotate -> matvec, each against its formula, and the chain from the normalised row on: the rotated row is
    within e ||x||_group of the exact one (half a step of each element at most), so y moves by at most e sum_g ||x||_group ||W||_group."""
    b = Block(710)
    att, stream = b.inputs(M, M)
    w = [v.to(dtype) for v in b.w]
    h, hs = pq.block_norms(att, stream, w[0], None, w[1])
    tn._check(f"norms {dtype}", (h, hs), tn._reference(att, stream, w[0], None, 1e-6, 1.0, 1.0, "none", False), w[1], 1e-6, False)
    rec, cs = b.rot["in"]
    x = pq.rotate(hs, rec, cs)
    layer = tm.Layer(K, 2048, 720)
    y = pq.matvec(x, layer.wpk, layer.sz, 2048)
    tm._check(f"chain {dtype}", y, x, layer, [(0, 2048)])
    # end to end, the rotation in 64 bits
    import test_rotate as tr
    from oracle import records as orec
    pl, tl, cl = synth.rotations(synth.Workload("ffn", 710, 1, K, 128))
    v, norm = tr._rotate64(hs.float().cpu().numpy(), orec.build(pl[0], tl[0]), cl[0])
    v, norm = torch.from_numpy(v).cuda(), torch.from_numpy(norm).cuda()
    ref = v @ layer.W
    e = torch.finfo(dtype).eps / 2
    moved = (e * v.abs() + 1.01 * 36 * tr.U * norm + 2.0 ** -25) @ layer.W.abs()
    bound = e * ref.abs() + (1 + e) * (moved + (256 + 3 * layer.G + 16) * tm.U * (v.abs() @ layer.mag) * (1 + 2 * e)) + 2.0 ** -25
    ratio = ((y.double() - ref).abs() / bound).max().item()
    print(f"[ffn 16-bit M={M}] end to end worst error/bound {ratio:.3f}", flush=True)
    assert ratio <= 1.0


def test_captured_block_replays_with_new_inputs():
    """The whole half captured once, replayed on new inputs, with eager steps of another block between the replays."""
    b, other = Block(), Block(730, F=1040)
    for M in (2, 40):
        att, stream = b.inputs(M, 1)
        k = {}
        b.forward(att, stream, k)                       # allocates every buffer
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            b.forward(att, stream, k)
        for r in range(3):
            new = b.inputs(M, 10 + r)
            att.copy_(new[0])
            stream.copy_(new[1])
            g.replay()
            other.forward(*other.inputs(M + 1, r), {})
            want = {}
            b.forward(*new, want)
            torch.cuda.synchronize()
            for name in ("stream1", "hs", "h", "y", "stream2", "hs2"):
                assert torch.equal(k[name], want[name]), (M, r, name)


def test_two_streams_at_once():
    """Two blocks on two streams, their calls interleaved, each with its own buffers: the results of either alone."""
    b, c = Block(), Block(740)
    want = [blk.forward(*blk.inputs(33, 3), {}) for blk in (b, c)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream(), torch.cuda.Stream()], []
    data = [blk.inputs(33, 3) for blk in (b, c)]
    torch.cuda.synchronize()
    for s, blk, d in zip(streams, (b, c), data):
        with torch.cuda.stream(s):
            got.append([blk.forward(*d, {}) for _ in range(5)][-1])
    torch.cuda.synchronize()
    for (a1, a2), (b1, b2) in zip(want, got):
        assert torch.equal(a1, b1) and torch.equal(a2, b2)
