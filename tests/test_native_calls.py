"""The compiled calls of rotate, matvec, gemm_glu and block_norms against the same calls through Python: which calls they take,
the same bits, the same refusals (GPU); objects that are no tensors (CPU)."""
import os

import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth

gpu = pytest.mark.gpu


@pytest.fixture
def through_python():
    """Runs a call with the compiled calls switched off."""
    def run(f):
        pq._native()
        saved, pq._fast = pq._fast, False
        try:
            return f()
        finally:
            pq._fast = saved
    return run


def test_built_and_bound():
    assert os.path.exists(os.path.join(os.path.dirname(pq.__file__), "_binding.so")) and pq._native()


def test_anything_else_is_left_to_python():
    b, t = pq._native(), torch.zeros(4, 256, dtype=torch.float16)
    for v in (None, 1, "x", t, [t]):
        assert b.rotate(v, v, v, v) is NotImplemented
        assert b.matvec(v, v, v, 64, 64, 64, None, None) is NotImplemented
        assert b.gemm_glu(v, v, v, v, v, 64, 0, None, None, None, False) is NotImplemented
        assert b.block_norms(v, v, v, v, v, 1e-6, 1.0, 1.0, 0, False, None, None) is NotImplemented
    assert b.rotate() is NotImplemented and b.matvec(t) is NotImplemented and b.gemm_glu(t) is NotImplemented and b.block_norms(t) is NotImplemented
    for n in (2 ** 31, -2 ** 31 - 1, 2 ** 70, 1.5, None, "1"):
        assert b.matvec(t, t, t, n, 64, 64, None, None) is NotImplemented
        assert b.gemm_glu(t, t, t, t, t, n, 0, None, None, None, False) is NotImplemented


# ------------------------------------------------------------------------------------------
def _world():
    M, K, F, G = 6, 256, 128, 2   # a partition begins on a 128-column line
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")                                    # noqa: E731
    u8 = lambda *s: torch.randint(0, 120, s, generator=g, device="cuda").to(torch.uint8)          # noqa: E731
    word = lambda r: torch.randint(-2 ** 31, 2 ** 31 - 1, (r, F // 4), generator=g, device="cuda").to(torch.int32)   # noqa: E731
    wpk, sz = pq.pack_weights(word(K), word(G), rnd(G, 2 * F).abs().half())
    pairs, theta, _ = synth.rotations(synth.Workload("calls", 9, M, K, 2 * F))
    rec = torch.from_numpy(pq.build_records(pairs[0], theta[0])).cuda()
    return dict(M=M, K=K, F=F, G=G, x=rnd(M, K).half(), rec=rec, rec2=torch.stack([rec, rec]), cs=rnd(2, K).half(), A=u8(2, M, K), S=rnd(2, M, G).abs(),
                R=rnd(2, M, G), wpk=wpk, sz=sz, res=rnd(M, K), w=rnd(K).half(), v=rnd(K).half(), b=rnd(M, K).bfloat16(), gt=rnd(M, 1).half(),
                ws=torch.empty(max(16, pq.gemm_workspace_bytes(40, 2 * F, K)), dtype=torch.uint8, device="cuda"), A40=u8(1, 40, K), S40=rnd(1, 40, G).abs(),
                R40=rnd(1, 40, G))


def _calls(w):
    """Name -> the call, for every way the compiled calls take."""
    x, wpk, sz, N, F, h, bf = w["x"], w["wpk"], w["sz"], 2 * w["F"], w["F"], torch.float16, torch.bfloat16
    wide = torch.zeros(w["M"], w["K"] + 8, dtype=h, device="cuda")
    wide[:, :w["K"]] = x
    xs, M, K = wide[:, :w["K"]], w["M"], w["K"]
    new = lambda *s, dtype=h: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    return {
        "rotate": lambda: pq.rotate(x, w["rec"], w["cs"][0]),
        "rotate, one partition in 2-D": lambda: pq.rotate(xs, w["rec"], w["cs"][:1]),
        "rotate, partitions": lambda: pq.rotate(w["b"], w["rec2"], w["cs"], out=new(2, M, K, dtype=bf)),
        "rotate, records [1, ..], scales [K]": lambda: pq.rotate(x, w["rec"][None], w["cs"][0]),
        "rotate, no rows": lambda: pq.rotate(x[:0], w["rec"], w["cs"][0]),
        "matvec": lambda: pq.matvec(x, wpk, sz, N),
        "matvec, rows apart, bf16": lambda: pq.matvec(xs, wpk, sz, N, dtype=bf),
        "matvec, partitions, out": lambda: pq.matvec(torch.stack([x, x + 1]), wpk, sz, N, F, N, out=new(M, N + 4)[:, :N]),
        "matvec, one row": lambda: pq.matvec(w["b"][:1], wpk, sz, N, out=new(1, N, dtype=h), dtype=h),
        "gemm_glu": lambda: pq.gemm_glu(w["A"][:1], w["S"][:1], w["R"][:1], wpk, sz, F),
        "gemm_glu, gelu, out": lambda: pq.gemm_glu(w["A"], w["S"], w["R"], wpk, sz, F, act="gelu", out=new(M, F + 2, dtype=bf)[:, :F]),
        "gemm_glu, own workspace": lambda: pq.gemm_glu(w["A40"], w["S40"], w["R40"], wpk, sz, F, dtype=bf),
        "gemm_glu, workspace": lambda: pq.gemm_glu(w["A40"], w["S40"], w["R40"], wpk, sz, F, workspace=w["ws"]),
        "block_norms": lambda: pq.block_norms(x, w["res"], w["w"], None, w["v"]),
        "block_norms, channel gate": lambda: pq.block_norms(x, w["res"], w["w"], w["v"], w["v"], gate_act="tanh", gemma=True, scale=2),
        "block_norms, token gate": lambda: pq.block_norms(x, w["res"].bfloat16(), None, w["gt"], w["v"], gate_act="sigmoid"),
        "block_norms, gate rows, no pre-norm": lambda: pq.block_norms(x, w["res"].half(), w["w"], xs, None, res_scale=0.5),
        "block_norms, out": lambda: pq.block_norms(xs, w["res"], None, None, w["v"], residual_out=new(M, K, dtype=torch.float32), out=new(M, K)),
        "block_norms, whole numbers": lambda: pq.block_norms(x, w["res"].clone(), w_pre=w["v"], eps=1),
    }


@gpu
def test_usual_calls_bypass_python_with_the_same_bits(through_python, monkeypatch):
    w = _world()
    for name, call in _calls(w).items():
        want = through_python(call)
        with monkeypatch.context() as m:
            m.setattr(pq, "_launch", None)      # the Python function's own launch would raise
            got = call()
        for a, b in zip(want if isinstance(want, tuple) else (want,), got if isinstance(got, tuple) else (got,)):
            assert (a is None) == (b is None), name
            if a is not None:
                assert a.dtype == b.dtype and a.shape == b.shape and a.device == b.device and torch.equal(a, b), name
    y = torch.empty_like(w["x"])[None]
    assert pq.rotate(w["x"], w["rec"], w["cs"][0], out=y) is y
    h, hs = torch.empty_like(w["res"]), torch.empty_like(w["x"])
    got = pq.block_norms(w["x"], w["res"], w_pre=w["v"], residual_out=h, out=hs)
    assert got[0] is h and got[1] is hs


@gpu
def test_refusals_are_the_same(through_python):
    w = _world()
    x, wpk, sz, F, cs, A, S, R = w["x"], w["wpk"], w["sz"], w["F"], w["cs"], w["A"], w["S"], w["R"]
    N, host = 2 * F, x.cpu()
    new = lambda *s, dtype=torch.float16: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    odd = new(w["M"] * w["K"] + 1)[1:].view(w["M"], w["K"])                            # off the 16-byte lines
    sub = torch.Tensor._make_subclass(type("T", (torch.Tensor,), {}), x)
    calls = [
        lambda: pq.rotate(host, w["rec"], cs[0]), lambda: pq.rotate(x.float(), w["rec"], cs[0]), lambda: pq.rotate(x[0], w["rec"], cs[0]),
        lambda: pq.rotate(x.t(), w["rec"], cs[0]), lambda: pq.rotate(x[:, :200], w["rec"], cs[0]), lambda: pq.rotate(x, w["rec"], cs),
        lambda: pq.rotate(x, w["rec2"], cs[:1]), lambda: pq.rotate(x, w["rec"], cs[0].float()), lambda: pq.rotate(x, w["rec"][:, :64], cs[0]),
        lambda: pq.rotate(x, w["rec"], cs[0], out=x[None]), lambda: pq.rotate(x, w["rec"], cs[0], out=new(6, 256)), lambda: pq.rotate(x, w["rec"], cs[0], out=odd[None]),
        lambda: pq.rotate(x[:1].expand(6, 256), w["rec"], cs[0]), lambda: pq.rotate(x[:, :0], w["rec"], cs[0]), lambda: pq.rotate(x.to_sparse(), w["rec"], cs[0]),
        lambda: pq.matvec(x, wpk, sz, N + 8), lambda: pq.matvec(x, wpk, sz, N + 16), lambda: pq.matvec(x, wpk, sz, -16), lambda: pq.matvec(x, wpk[16:], sz, N),
        lambda: pq.matvec(x, wpk, sz.float(), N), lambda: pq.matvec(x, wpk, sz[:1], N), lambda: pq.matvec(x.repeat(3, 1), wpk, sz, N),
        lambda: pq.matvec(x[:, 1:], wpk, sz, N), lambda: pq.matvec(x, wpk, sz, N, 32, 64), lambda: pq.matvec(x[None], wpk, sz, N, out=new(6, N - 16)),
        lambda: pq.matvec(x, wpk, sz, N, out=new(6, N), dtype=torch.bfloat16), lambda: pq.matvec(x, wpk, sz, N, dtype=torch.float32),
        lambda: pq.matvec(x, wpk, sz, N, out=new(N, 6).t()), lambda: pq.matvec(x, wpk, sz, N, out=new(1, N).expand(6, N)), lambda: pq.matvec(odd, wpk, sz, N),
        lambda: pq.matvec(x[None].expand(2, 6, 256), wpk, sz, N, F, N), lambda: pq.matvec(x.double(), wpk, sz, N), lambda: pq.matvec(x, wpk, sz, N, out=new(6, N + 1)),
        lambda: pq.matvec(x, wpk, sz, float(N)), lambda: pq.matvec(x, wpk, sz, N, out=host),
        lambda: pq.gemm_glu(A[0], S, R, wpk, sz, F), lambda: pq.gemm_glu(A, S[:1], R, wpk, sz, F), lambda: pq.gemm_glu(A, S, R.half(), wpk, sz, F),
        lambda: pq.gemm_glu(A, S, R, wpk, sz, F, act="relu"), lambda: pq.gemm_glu(A, S, R, wpk, sz, F, act=None), lambda: pq.gemm_glu(A, S, R, wpk, sz, F + 8),
        lambda: pq.gemm_glu(A, S, R, wpk, sz, -F), lambda: pq.gemm_glu(A, S, R, wpk, sz, 2 * F), lambda: pq.gemm_glu(A, S, R, wpk, sz, F, dtype=torch.float32),
        lambda: pq.gemm_glu(w["A40"], w["S40"], w["R40"], wpk, sz, F, prepared=True), lambda: pq.gemm_glu(w["A40"], w["S40"], w["R40"], wpk, sz, F, workspace=w["ws"][:64]),
        lambda: pq.gemm_glu(w["A40"], w["S40"], w["R40"], wpk, sz, F, workspace=w["ws"][1:]), lambda: pq.gemm_glu(A, S, R, wpk, sz, F, out=new(6, F, dtype=torch.float32)),
        lambda: pq.gemm_glu(torch.cat([A, A]), torch.cat([S, S]), torch.cat([R, R]), wpk, sz, F),
        lambda: pq.block_norms(x, host), lambda: pq.block_norms(x, w["res"][:3]), lambda: pq.block_norms(x, w["res"], w["w"].bfloat16(), None, w["v"]),
        lambda: pq.block_norms(x, w["res"], gate=w["b"]), lambda: pq.block_norms(x, w["res"], gate=w["v"][:8]), lambda: pq.block_norms(x, w["res"], gate=w["gt"][:3]),
        lambda: pq.block_norms(x, w["res"], gate=w["v"][None]), lambda: pq.block_norms(x, w["res"], out=x), lambda: pq.block_norms(x, w["res"], w_pre=w["v"], out=x),
        lambda: pq.block_norms(x, w["res"], eps=0.0), lambda: pq.block_norms(x, w["res"], eps=None), lambda: pq.block_norms(x, w["res"], gate_act="relu"),
        lambda: pq.block_norms(odd, w["res"]), lambda: pq.block_norms(x, w["res"], residual_out=w["res"][:, :128]), lambda: pq.block_norms(x, w["res"].double()),
        lambda: pq.block_norms(x[:, :12], w["res"][:, :12]), lambda: pq.block_norms(x, x, residual_out=x), lambda: pq.block_norms(sub, host),
    ]
    for i, call in enumerate(calls):
        said = []
        for run in (through_python, lambda f: f()):
            with pytest.raises(Exception) as e:
                run(call)
            said.append((type(e.value), str(e.value)))
        assert said[0] == said[1], (i, said)
    torch.cuda.synchronize()


@gpu
def test_subclass_parameter_and_streams(through_python):
    w = _world()
    x, want = w["x"], pq.matvec(w["x"], w["wpk"], w["sz"], 2 * w["F"])
    sub = torch.Tensor._make_subclass(type("T", (torch.Tensor,), {}), x)
    for v in (sub, torch.nn.Parameter(x), torch.nn.Parameter(x, requires_grad=False)):
        y = pq.matvec(v, w["wpk"], w["sz"], 2 * w["F"])
        assert torch.equal(y, want) and not y.requires_grad
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = pq.matvec(x, w["wpk"], w["sz"], 2 * w["F"])
    b = pq.matvec(x, w["wpk"], w["sz"], 2 * w["F"], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, want) and torch.equal(b, want)
    with torch.inference_mode():
        assert torch.equal(pq.matvec(x, w["wpk"], w["sz"], 2 * w["F"]), want)


@gpu
def test_two_threads_and_a_graph():
    """Calls from two Python threads on streams of their own, and captured with their outputs made in the capture, replayed between eager calls."""
    import threading
    w = _world()
    calls = [c for n, c in _calls(w).items() if "no rows" not in n and "whole numbers" not in n]
    flat = lambda r: [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]   # noqa: E731
    want = [[t.clone() for t in flat(c())] for c in calls]
    torch.cuda.synchronize()
    failed = []

    def work():
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(20):
                for c, ref in zip(calls, want):
                    if not all(torch.equal(a, b) for a, b in zip(flat(c()), ref)):
                        failed.append(1)
        s.synchronize()
    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [flat(c()) for c in calls]
    for _ in range(3):
        for o in outs:
            for t in o:
                t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, ref in zip(outs, want) for a, b in zip(o, ref))
        assert all(torch.equal(a, b) for c, ref in zip(calls, want) for a, b in zip(flat(c()), ref))
