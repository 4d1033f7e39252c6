"""A call's status is that of its own launches. An error that other code left in the thread (here: a device that does not
exist, asked for through the runtime) is neither taken for a failed launch nor cleared; a launch that fails is reported."""
import ctypes

import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth


def _runtime():
    """The HIP runtime that this process has loaded."""
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
    assert len(paths) == 1, paths
    return ctypes.CDLL(paths.pop())


def _calls():
    """Every entry point that launches, into outputs made before."""
    M, K, F = 40, 256, 128
    N = 2 * F
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")                                                        # noqa: E731
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=g, device="cuda").to(torch.int32)             # noqa: E731
    new = lambda *s, dtype=torch.float16: torch.zeros(s, dtype=dtype, device="cuda")                                   # noqa: E731
    qw, qz, sc = words(K, N // 8), words(2, N // 8), rnd(2, N).abs().half()
    qwh, qzh = words(K, N // 32), words(2, N // 32)
    wpk, sz = pq.pack_weights(qw, qz, sc)
    wpk5, sz5 = pq.pack_weights5(qw, qwh, qz, qzh, sc)
    pairs, theta, _ = synth.rotations(synth.Workload("status", 9, M, K, N))
    rec, cs = torch.from_numpy(pq.build_records(pairs[0], theta[0])).cuda(), rnd(1, K).half()
    x, res, w = rnd(M, K).half(), rnd(M, K).half(), rnd(K).half()
    q = [new(1, M, K, dtype=torch.uint8), new(1, M, 2, dtype=torch.float32), new(1, M, 2, dtype=torch.float32)]
    qi = [new(1, M, K, dtype=torch.int8), q[1].clone(), q[2].clone()]
    qt = [new(1, M, K, dtype=torch.uint8), new(1, M, dtype=torch.float32), q[2].clone()]
    codes, codes_i, codes_t = pq.rotate_quant(x, rec, cs), pq.rotate_quant_i8(x, rec, cs), pq.rotate_quant_tok(x, rec, cs)
    few = tuple(t[:, :5].contiguous() for t in codes)
    big = pq.pack_weights(words(K, 2 * 8704 // 8), words(2, 2 * 8704 // 8), rnd(2, 2 * 8704).abs().half())
    many = tuple(t.repeat(1, 30, 1) for t in codes)
    ws = new(max(pq.gemm_workspace_bytes(1200, N, K), pq.gemm_tok_workspace_bytes(M, N, K)), dtype=torch.uint8)
    y, h, hm = new(M, N, dtype=torch.bfloat16), new(M, F), new(1200, 8704)
    prod = [new(M, K), *[t.clone() for t in q]]
    f32 = rnd(100)
    return {
        "rotate": (lambda: pq.rotate(x, rec, cs, out=prod[0][None]), prod[:1]),
        "matvec": (lambda: pq.matvec(x[:5], wpk, sz, N, out=h.view(-1)[:5 * N].view(5, N)), [h]),
        "gemm_glu, few rows": (lambda: pq.gemm_glu(*few, wpk, sz, F, out=h[:5]), [h]),
        "gemm_glu, row blocks": (lambda: pq.gemm_glu(*codes, wpk, sz, F, out=h, workspace=ws), [h]),
        "gemm_glu, tiles": (lambda: pq.gemm_glu(*many, *big, 8704, out=hm, workspace=ws), [hm]),
        "block_norms": (lambda: pq.block_norms(x, res, w, None, w, residual_out=prod[0], out=hm.view(-1)[:M * K].view(M, K)),
                        [prod[0], hm]),
        "rotate_quant": (lambda: pq.rotate_quant(x, rec, cs, out=q), q),
        "rotate_quant_for_gemm": (lambda: pq.rotate_quant_for_gemm(x, rec, cs, ws, out=q), q),
        "rotate_quant_i8": (lambda: pq.rotate_quant_i8(x, rec, cs, out=qi), qi),
        "rotate_quant_tok": (lambda: pq.rotate_quant_tok(x, rec, cs, out=qt), qt),
        "add_rms_rotate_quant": (lambda: pq.add_rms_rotate_quant(x, res, w, 1e-6, rec, cs, residual_out=y.view(torch.float16)[:, :K], out=prod), [y, *prod]),
        "gemm": (lambda: pq.gemm(*codes, wpk, sz, N, out=y, workspace=ws), [y]),
        "gemm, few rows": (lambda: pq.gemm(*few, wpk, sz, N, out=y[:5]), [y]),
        "gemm_i8": (lambda: pq.gemm_i8(*codes_i, wpk, sz, N, out=y, workspace=ws), [y]),
        "gemm_tok": (lambda: pq.gemm_tok(*codes_t, wpk, sz, N, out=y, workspace=ws), [y]),
        "gemm5": (lambda: pq.gemm5(*codes, wpk5, sz5, N, out=y, workspace=ws), [y]),
        "gemm_noalloc": (lambda: pq.gemm_noalloc(*codes, wpk, sz, N, out=y), [y]),
        "pack_weights": (lambda: pq.pack_weights(qw, qz, sc), []),
        "pack_weights5": (lambda: pq.pack_weights5(qw, qwh, qz, qzh, sc), []),
        "e4m3_encode": (lambda: pq.e4m3_encode(f32), []),
        "recip_f32": (lambda: pq.recip_f32(f32), []),
        "bf16_round": (lambda: pq.bf16_round(f32), []),
    }


@pytest.mark.gpu
def test_an_error_left_by_other_code_is_not_the_calls():
    hip = _runtime()
    for name, (call, outs) in _calls().items():
        print(f"[status] {name}", flush=True)
        for t in outs:
            t.zero_()
        call()
        torch.cuda.synchronize()
        want = [t.clone() for t in outs]
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        assert hip.hipSetDevice(4096) != 0
        left = hip.hipPeekAtLastError()
        try:
            call()
        finally:
            after = hip.hipGetLastError()     # torch's own checks would report it at the next operation
        torch.cuda.synchronize()
        assert after == left, name
        for a, b in zip(want, outs):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="the addresses are not real: only where nothing can be launched")
def test_a_launch_that_fails_is_reported():
    """Without a device every launch fails: the code and the message say so, from the first of a call's launches on."""
    L, at = pq.lib(), 1 << 32
    p = [at + (i << 24) for i in range(12)]
    calls = [
        L.pq_rotate(p[0], 256, 0, 4, 256, 1, p[1], p[2], p[3], None), L.pq_matvec(p[0], 256, 0, 4, 256, 1, p[1], p[2], 128, *[pq.NO_BOUNDARY] * 2, p[3], 128, 0, None),
        L.pq_block_norms(p[0], 256, 0, p[1], 256, 0, p[2], None, 0, 256, 0, p[3], 1e-6, 1.0, 1.0, 0, 4, 256, p[4], 256, p[5], 256, 0, None),
        L.pq_gemm_glu(p[0], p[1], p[2], 4, 256, 1, p[3], p[4], 64, 0, p[5], 64, 0, None, 0, 0, None),
        L.pq_gemm_glu(p[0], p[1], p[2], 40, 256, 1, p[3], p[4], 64, 0, p[5], 64, 0, p[6], 1 << 24, 0, None),
        L.pq_gemm_glu(p[0], p[1], p[2], 1200, 256, 1, p[3], p[4], 8704, 0, p[5], 8704, 0, p[8], 1 << 24, 0, None),
        L.pq_gemm(p[0], p[1], p[2], 40, 256, 1, p[3], p[4], 64, *[pq.NO_BOUNDARY] * 2, p[5], 64, p[6], 1 << 24, None),
        L.pq_rotate_quant(p[0], 256, 4, 256, 1, p[1], p[2], p[3], p[4], p[5], None), L.pq_pack_weights(p[0], p[1], p[2], 256, 64, p[3], p[4], None)]
    assert calls == [-7] * len(calls)
    assert b"launch failed" in L.pq_last_error()
