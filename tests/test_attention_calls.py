"""kv_write, kv_read, attn_decode and attn_prefill as calls: the compiled calls against the same calls through Python (the same bits,
the same refusals), other streams, two threads, graphs, workspaces, what a call's status is, and sizes past 31 bits."""
import ctypes
import threading

import pytest
import torch

import rotated_w4a8_group_amd as pq

gpu = pytest.mark.gpu
F16, BF16, U8, F32, I32, I64 = torch.float16, torch.bfloat16, torch.uint8, torch.float32, torch.int32, torch.int64


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


def test_anything_else_is_left_to_python():
    b, t = pq._native(), torch.zeros(4, 2, 128, dtype=F16)
    for v in (None, 1, "x", t, [t]):
        assert b.kv_write(v, v, v, v, v, v, v) is NotImplemented
        assert b.kv_read(v, v, v, v, 4, v, v, None, None) is NotImplemented
        assert b.attn_decode(v, v, v, v, v, v, v, None, None, None, None) is NotImplemented
        assert b.attn_prefill(v, v, v, v, None, None, True, None, None, None) is NotImplemented
    assert b.kv_write() is NotImplemented and b.kv_read(t) is NotImplemented and b.attn_decode(t) is NotImplemented and b.attn_prefill(t) is NotImplemented
    for n in (2 ** 31, -1, 2 ** 70, 1.5, None, "1"):
        assert b.kv_read(t, t, t, t, n, t, t, None, None) is NotImplemented


# ------------------------------------------------------------------------------------------
WRAP = 2 ** 32


def _e(*shape, dtype=F16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _decode_meta(B=2, Hq=8, Hkv=2, D=128, pages=3, page=16, width=3):
    return (_e(B, Hq, D), _e(pages, Hkv, page, D), _e(pages, Hkv, page, D), _e(B, width, dtype=I32), _e(B, dtype=I32))


LARGE = {
    "kv_write rows": lambda: pq.kv_write(_e(WRAP, 1, 128), _e(WRAP, 1, 128), _e(WRAP, dtype=I64), _e(1, 1, 16, 128), _e(1, 1, 16, 128)),
    "kv_write heads": lambda: pq.kv_write(_e(1, WRAP + 1, 128), _e(1, WRAP + 1, 128), _e(1, dtype=I64), _e(1, WRAP + 1, 16, 128), _e(1, WRAP + 1, 16, 128)),
    "kv_write pages": lambda: pq.kv_write(_e(1, 1, 128), _e(1, 1, 128), _e(1, dtype=I64), _e(WRAP, 1, 16, 128), _e(WRAP, 1, 16, 128)),
    "kv_read rows": lambda: pq.kv_read(_e(1, 1, 16, 128), _e(1, 1, 16, 128), _e(1, 1, dtype=I32), _e(2, dtype=I32), WRAP + 1),
    "kv_read width": lambda: pq.kv_read(_e(1, 1, 16, 128), _e(1, 1, 16, 128), _e(1, WRAP + 1, dtype=I32), _e(2, dtype=I32), 4),
    "attn_decode sequences": lambda: pq.attn_decode(*_decode_meta(B=WRAP)),
    "attn_decode heads": lambda: pq.attn_decode(*_decode_meta(Hq=WRAP + 8)),
    "attn_decode pages": lambda: pq.attn_decode(*_decode_meta(pages=WRAP)),
    "attn_decode width": lambda: pq.attn_decode(*_decode_meta(width=WRAP + 1)),
    "attn_prefill rows": lambda: pq.attn_prefill(_e(WRAP, 1, 128), _e(1, 1, 128), _e(1, 1, 128), _e(2, dtype=I32)),
    "attn_prefill keys": lambda: pq.attn_prefill(_e(1, 1, 128), _e(WRAP, 1, 128), _e(WRAP, 1, 128), _e(2, dtype=I32)),
    "attn_prefill sequences": lambda: pq.attn_prefill(_e(1, 1, 128), _e(1, 1, 128), _e(1, 1, 128), _e(WRAP, dtype=I32)),
    "workspace of an attn_decode": lambda: pq.attn_decode_workspace_bytes(WRAP + 1, 8, 2, 128),
    "workspace of an attn_prefill": lambda: pq.attn_prefill_workspace_bytes(1, 64, WRAP + 64, 8, 2, 128),
}


@pytest.mark.parametrize("name", LARGE)
def test_sizes_past_31_bits(name):
    with pytest.raises(ValueError, match="at most 2\\^31 - 1 in one call"):
        LARGE[name]()


@pytest.mark.parametrize("B,width,page,Hq,Hkv,code", [
    (1, 2 ** 21, 1024, 8, 8, -2),            # 2^31 positions
    (2 ** 12, 2 ** 17, 256, 64, 64, -2),     # 2^38 tiles
    (1, 2 ** 21 - 1, 1024, 32, 32, -2),      # 2^31 tiles, and the pieces' rounding past them
    (2 ** 16, 16, 16, 16, 16, -6),           # passes these checks: the workspace is next
])
def test_decode_tables_that_are_too_large(B, width, page, Hq, Hkv, code):
    at = [(1 << 44) + (i << 40) for i in range(9)]
    L = pq.lib()
    rc = L.pq_attn_decode(at[0], Hq * 128, 128, 1, at[1], at[2], at[3], at[4], 9, page, at[5], width, at[6], B, Hq, Hkv, 128, 0.1, at[7], 0, at[8], 16, None)
    assert rc == code


def test_workspaces_that_are_too_small():
    L, at = pq.lib(), [(1 << 44) + (i << 40) for i in range(9)]
    need = pq.attn_decode_workspace_bytes(2, 48, 8, 128)
    assert need > 0
    for ws, n, code in ((None, need, -6), (at[8], need - 1, -6), (at[8] + 8, need, -3)):
        assert L.pq_attn_decode(at[0], 6144, 128, 1, at[1], at[2], at[3], at[4], 9, 16, at[5], 300, at[6], 2, 48, 8, 128, 0.1, at[7], 0, ws, n, None) == code
    need = pq.attn_prefill_workspace_bytes(1, 40, 9000, 8, 2, 128)
    assert need > 0 and pq.attn_prefill_workspace_bytes(1, 9000, 9000, 48, 8, 128) == 0
    for ws, n, code in ((None, need, -6), (at[8], need - 1, -6), (at[8] + 8, need, -3)):
        assert L.pq_attn_prefill(at[0], 1024, 128, at[1], 256, 128, at[2], 256, 128, 1, at[3], at[4], 1, 40, 9000, 8, 2, 128, 0.1, 1, at[5], 0, ws, n, None) == code


# ------------------------------------------------------------------------------------------
def _world(seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")                                    # noqa: E731
    T, Hq, Hkv, D, page, pages, B = 70, 12, 2, 128, 16, 90, 3
    y = rnd(T, (Hq + 2 * Hkv) * D).bfloat16()
    q, k, v = y[:, :Hq * D].unflatten(1, (Hq, D)), y[:, Hq * D:(Hq + Hkv) * D].unflatten(1, (Hkv, D)), y[:, (Hq + Hkv) * D:].unflatten(1, (Hkv, D))
    cache = [torch.zeros((pages, Hkv, page, D), dtype=U8, device="cuda") for _ in range(2)] + [torch.zeros((pages, Hkv, page), device="cuda") for _ in range(2)]
    half = [rnd(pages, Hkv, page, D).bfloat16() for _ in range(2)]
    slots = torch.randperm(pages * page, generator=g, device="cuda")
    pq.kv_write(rnd(pages * page, Hkv, D).bfloat16(), rnd(pages * page, Hkv, D).bfloat16(), slots, *cache)
    table = torch.randperm(pages, generator=g, device="cuda")[:81].to(I32).reshape(B, 27).repeat(1, 4).contiguous()   # up to 1728 positions
    lens = torch.tensor([1700, 33, 900], dtype=I32, device="cuda")
    cu = torch.tensor([0, 33, 33, 70], dtype=I32, device="cuda")
    long = rnd(2000, 2 * Hkv * D).bfloat16()
    cu_k = torch.tensor([0, 1900, 1900, 2000], dtype=I32, device="cuda")
    return dict(T=T, Hq=Hq, Hkv=Hkv, D=D, B=B, q=q, k=k, v=v, cache=cache, half=half, slots=slots[:T].contiguous(), table=table, lens=lens, cu=cu,
                kl=long[:, :Hkv * D].unflatten(1, (Hkv, D)), vl=long[:, Hkv * D:].unflatten(1, (Hkv, D)), cu_k=cu_k,
                ws=torch.empty(max(pq.attn_decode_workspace_bytes(B, Hq, Hkv, D), pq.attn_prefill_workspace_bytes(3, T, 2000, Hq, Hkv, D)), dtype=U8, device="cuda"))


def _calls(w):
    """Name -> the call, for every way the compiled calls take; those that write a cache write one of their own."""
    new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    T, Hq, Hkv, D, B, c, h = w["T"], w["Hq"], w["Hkv"], w["D"], w["B"], w["cache"], w["half"]
    own, own16 = [t.clone() for t in c], [t.clone() for t in h]
    qd, short = w["q"][:B], w["table"][:, :10].contiguous()
    total = int(w["lens"].sum())
    cu_r = torch.tensor([0, 1700, 1733, 2633], dtype=I32, device="cuda")
    return {
        "kv_write": lambda: (*pq.kv_write(w["k"], w["v"], w["slots"], *own), own[2], own[3]),
        "kv_write, one row": lambda: (*pq.kv_write(w["k"][:1], w["v"][:1], w["slots"][:1], *own), own[2], own[3]),
        "kv_write, 16-bit": lambda: pq.kv_write(w["k"], w["v"], w["slots"], *own16),
        "kv_write, no rows": lambda: pq.kv_write(w["k"][:0], w["v"][:0], w["slots"][:0], *own16),
        "kv_read": lambda: pq.kv_read(c[0], c[1], w["table"], cu_r, total, c[2], c[3]),
        "kv_read, bf16": lambda: pq.kv_read(c[0], c[1], w["table"], cu_r, total, c[2], c[3], dtype=BF16),
        "kv_read, 16-bit cache": lambda: pq.kv_read(h[0], h[1], w["table"], cu_r, total),
        "kv_read, out": lambda: pq.kv_read(c[0], c[1], w["table"], cu_r, total, c[2], c[3], out=(new(total, Hkv, D), new(total, Hkv, D))),
        "attn_decode": lambda: pq.attn_decode(qd, c[0], c[1], w["table"], w["lens"], c[2], c[3]),
        "attn_decode, short table": lambda: pq.attn_decode(qd, c[0], c[1], short, w["lens"], c[2], c[3], dtype=F16),
        "attn_decode, 16-bit cache, scale": lambda: pq.attn_decode(qd, h[0], h[1], w["table"], w["lens"], scale=0.05),
        "attn_decode, out": lambda: pq.attn_decode(qd, c[0], c[1], w["table"], w["lens"], c[2], c[3], scale=1, out=new(B, Hq, D, dtype=F16)),
        "attn_prefill": lambda: pq.attn_prefill(w["q"], w["k"], w["v"], w["cu"]),
        "attn_prefill, all keys": lambda: pq.attn_prefill(w["q"], w["k"], w["v"], w["cu"], causal=False, dtype=F16),
        "attn_prefill, long keys": lambda: pq.attn_prefill(w["q"], w["kl"], w["vl"], w["cu"], w["cu_k"]),
        "attn_prefill, out, scale": lambda: pq.attn_prefill(w["q"], w["kl"], w["vl"], w["cu"], w["cu_k"], scale=0.2, out=new(T, Hq, D)),
        "attn_prefill, no rows": lambda: pq.attn_prefill(w["q"][:0], w["k"][:0], w["v"][:0], w["cu"][:1]),
    }


def _with_workspace(w):
    """The calls that take a workspace, with one: for one call at a time."""
    c = w["cache"]
    return {"attn_decode": lambda: pq.attn_decode(w["q"][:w["B"]], c[0], c[1], w["table"], w["lens"], c[2], c[3], workspace=w["ws"]),
            "attn_prefill, long keys": lambda: pq.attn_prefill(w["q"], w["kl"], w["vl"], w["cu"], w["cu_k"], workspace=w["ws"])}


def _flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


@gpu
def test_usual_calls_bypass_python_with_the_same_bits(through_python, monkeypatch):
    w = _world()
    for calls in (_calls(w), _with_workspace(w)):
        for name, call in calls.items():
            want = [t.clone() for t in _flat(through_python(call))]
            with monkeypatch.context() as m:
                m.setattr(pq, "_launch", None)      # the Python function's own launch would raise
                got = _flat(call())
            for a, b in zip(want, got):
                assert a.dtype == b.dtype and a.shape == b.shape and torch.equal(a, b), name
    for name, call in _with_workspace(w).items():   # a workspace makes no difference, whatever it held
        w["ws"].fill_(0xFF)
        assert torch.equal(call(), _calls(w)[name]()), name
    o = torch.empty_like(w["q"][:3]).contiguous()
    assert pq.attn_decode(w["q"][:3], *w["cache"][:2], w["table"], w["lens"], *w["cache"][2:], out=o) is o


@gpu
def test_refusals_are_the_same(through_python):
    w = _world()
    c, h, q, k, v, table, lens, cu, slots = w["cache"], w["half"], w["q"], w["k"], w["v"], w["table"], w["lens"], w["cu"], w["slots"]
    new = lambda *s, dtype=F16: torch.empty(s, dtype=dtype, device="cuda")   # noqa: E731
    odd = new(70 * 256 + 1, dtype=BF16)[1:].view(70, 2, 128)                # off the 16-byte lines
    apart = new(70, 2, 132, dtype=BF16)[:, :, :128]                         # heads off them
    qd = q[:3]
    calls = [
        lambda: pq.kv_write(k.cpu(), v, slots, *c), lambda: pq.kv_write(k.float(), v, slots, *c), lambda: pq.kv_write(k, v.half(), slots, *c),
        lambda: pq.kv_write(k[:3], v, slots, *c), lambda: pq.kv_write(k, v, slots.int(), *c), lambda: pq.kv_write(k, v, slots[:5], *c),
        lambda: pq.kv_write(k, v, slots, c[0][:, :1], c[1], *c[2:]), lambda: pq.kv_write(k, v, slots, c[0], c[1]), lambda: pq.kv_write(k, v, slots, *c[:3]),
        lambda: pq.kv_write(k, v, slots, h[0].half(), h[1].half()), lambda: pq.kv_write(odd, v, slots, *c), lambda: pq.kv_write(apart, v, slots, *c),
        lambda: pq.kv_write(k[..., :64], v[..., :64], slots, *c), lambda: pq.kv_write(k.transpose(1, 2), v, slots, *c), lambda: pq.kv_write(k, v, slots, c[0].cpu(), *c[1:]),
        lambda: pq.kv_write(k[..., :32], v[..., :32], slots, h[0][..., :32].contiguous(), h[1][..., :32].contiguous()),
        lambda: pq.kv_read(c[0], c[1], table, cu, 70, *c[2:], dtype=F32), lambda: pq.kv_read(c[0], c[1], table, cu[:2], 70, *c[2:]),
        lambda: pq.kv_read(c[0], c[1], table.long(), cu, 70, *c[2:]), lambda: pq.kv_read(c[0], c[1], table, cu, -1, *c[2:]),
        lambda: pq.kv_read(c[0], c[1], table, cu, 70), lambda: pq.kv_read(h[0], h[1], table, cu, 70, dtype=F16),
        lambda: pq.kv_read(c[0], c[1], table, cu, 70, *c[2:], out=(new(70, 2, 128),)), lambda: pq.kv_read(c[0], c[1], table, cu, 70, *c[2:], out=(new(71, 2, 128), new(70, 2, 128))),
        lambda: pq.kv_read(c[0], c[1], table, cu, 70, *c[2:], out=(new(70, 2, 128), new(70, 2, 128, dtype=BF16))), lambda: pq.kv_read(c[0], c[1], table[:, 0], cu, 70, *c[2:]),
        lambda: pq.kv_read(c[0], c[1], table, cu, 70, *c[2:], out=(new(70, 2, 128), new(70, 2, 128)), dtype=BF16),
        lambda: pq.attn_decode(qd.cpu(), c[0], c[1], table, lens, *c[2:]), lambda: pq.attn_decode(q[:2], c[0], c[1], table, lens, *c[2:]),
        lambda: pq.attn_decode(qd[:, :11], c[0], c[1], table, lens, *c[2:]), lambda: pq.attn_decode(qd[..., :64], c[0], c[1], table, lens, *c[2:]),
        lambda: pq.attn_decode(qd, c[0], c[1], table, lens.long(), *c[2:]), lambda: pq.attn_decode(qd, c[0], c[1], table[:2], lens, *c[2:]),
        lambda: pq.attn_decode(qd.half(), h[0], h[1], table, lens), lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], scale=0.0),
        lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], scale=-1), lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], scale="x"),
        lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], out=new(3, 12, 64)), lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], out=new(3, 12, 128), dtype=BF16),
        lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], workspace=w["ws"][:100]), lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], workspace=w["ws"][8:]),
        lambda: pq.attn_decode(odd[:3].view(3, 2, 128), c[0], c[1], table, lens, *c[2:]), lambda: pq.attn_decode(qd, c[0], c[1], table, lens, *c[2:], dtype=F32),
        lambda: pq.attn_prefill(q.cpu(), k, v, cu), lambda: pq.attn_prefill(q, k.half(), v, cu), lambda: pq.attn_prefill(q, k[:5], v, cu), lambda: pq.attn_prefill(q[:, :11], k, v, cu),
        lambda: pq.attn_prefill(q, k, v, cu.long()), lambda: pq.attn_prefill(q, k, v, cu[:0]), lambda: pq.attn_prefill(q, k, v, cu, cu[:3]), lambda: pq.attn_prefill(q, k, v, cu[None]),
        lambda: pq.attn_prefill(q, odd, v, cu), lambda: pq.attn_prefill(q, k, apart, cu), lambda: pq.attn_prefill(q, k, v, cu, scale=float("nan")),
        lambda: pq.attn_prefill(q, k, v, cu, out=new(70, 12, 64)), lambda: pq.attn_prefill(q, k, v, cu, dtype=F32), lambda: pq.attn_prefill(q, k, v, cu, scale=None, out=q),
        lambda: pq.attn_prefill(q, w["kl"], w["vl"], cu, w["cu_k"], workspace=w["ws"][:16]), lambda: pq.attn_prefill(q[..., :32], k[..., :32], v[..., :32], cu),
        lambda: pq.attn_prefill(*(new(0, 1, WRAP + 128) for _ in range(3)), cu),
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
def test_streams_subclasses_and_inference_mode():
    w = _world()
    calls, s = _calls(w), torch.cuda.Stream()
    want = {n: [t.clone() for t in _flat(f())] for n, f in calls.items()}
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = {n: [t.clone() for t in _flat(f())] for n, f in calls.items()}
    c = w["cache"]
    a = pq.attn_decode(w["q"][:3], c[0], c[1], w["table"], w["lens"], c[2], c[3], stream=s)
    b = pq.attn_prefill(w["q"], w["kl"], w["vl"], w["cu"], w["cu_k"], stream=s)
    k, v = pq.kv_read(c[0], c[1], w["table"], torch.tensor([0, 1700, 1733, 2633], dtype=I32, device="cuda"), 2633, c[2], c[3], stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for n in want:
        assert all(torch.equal(x, y) for x, y in zip(want[n], got[n])), n
    assert torch.equal(a, want["attn_decode"][0]) and torch.equal(b, want["attn_prefill, long keys"][0]) and torch.equal(k, want["kv_read"][0]) and torch.equal(v, want["kv_read"][1])
    sub = torch.Tensor._make_subclass(type("T", (torch.Tensor,), {}), w["q"][:3])
    for q in (sub, torch.nn.Parameter(w["q"][:3])):
        o = pq.attn_decode(q, c[0], c[1], w["table"], w["lens"], c[2], c[3])
        assert torch.equal(o, want["attn_decode"][0]) and not o.requires_grad
    with torch.inference_mode():
        assert torch.equal(pq.attn_prefill(w["q"], w["k"], w["v"], w["cu"]), want["attn_prefill"][0])


@gpu
@pytest.mark.parametrize("native", [True, False])
def test_two_threads(native):
    """Each on a stream of its own, with caches and workspaces of its own."""
    worlds = [_world(5), _world(6)]
    saved = pq._fast
    try:
        pq._native()
        if not native:
            pq._fast = False
        calls = [list(_calls(w).items()) + list(_with_workspace(w).items()) for w in worlds]
        want = [[[t.clone() for t in _flat(f())] for _, f in c] for c in calls]
        torch.cuda.synchronize()
        failed = []

        def work(i):
            try:
                s = torch.cuda.Stream()
                with torch.cuda.stream(s):
                    for _ in range(10):
                        for (n, f), ref in zip(calls[i], want[i]):
                            assert all(torch.equal(a, b) for a, b in zip(_flat(f()), ref)), n
                s.synchronize()
            except BaseException as e:   # noqa: B902
                failed.append(repr(e))
        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
    finally:
        pq._fast = saved
    assert not failed, failed[0]


@gpu
def test_captured_calls():
    """Captured together, workspaces made in the capture among them, replayed between eager calls."""
    w = _world()
    calls = [f for n, f in _calls(w).items() if "no rows" not in n]
    want = [[t.clone() for t in _flat(f())] for f in calls]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [_flat(f()) for f in calls]
    for _ in range(3):
        for o, f in zip(outs, calls):
            for t in o:
                t.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for o, ref in zip(outs[3:], want[3:]) for a, b in zip(o, ref))
        assert all(torch.equal(a, b) for f, ref in zip(calls[3:], want[3:]) for a, b in zip(_flat(f()), ref))


@gpu
def test_replays_follow_lengths_and_pages():
    """A served model replays one graph while its sequences grow and change pages: the eager call's bits at every step."""
    w = _world()
    c, table, lens, cu, cu_k = w["cache"], w["table"].clone(), w["lens"].clone(), w["cu"].clone(), w["cu_k"].clone()
    calls = [lambda: pq.attn_decode(w["q"][:3], c[0], c[1], table, lens, c[2], c[3]), lambda: pq.attn_prefill(w["q"], w["kl"], w["vl"], cu, cu_k),
             lambda: pq.attn_prefill(w["q"], w["k"], w["v"], cu)]
    for f in calls:
        f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        outs = [f() for f in calls]
    for step in ([1, 1, 1], [0, 1728, 0], [300, 301, 1727], [1728, 1728, 1728], [5, 0, 64], [0, 0, 0]):
        lens.copy_(torch.tensor(step))
        table.copy_(table.flip(0).roll(1, 1))
        a, b = sorted(n % 71 for n in step[:2])
        cu.copy_(torch.tensor([0, a, b, 70]))
        cu_k.copy_(torch.tensor([0, 70 + step[0], 70 + step[0], 2000]))
        for o in outs:
            o.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        for o, f in zip(outs, calls):
            assert torch.equal(o, f()), step


@gpu
def test_two_graphs_with_one_workspace():
    """One after the other they may share a workspace: a call takes nothing from what it holds."""
    w = _world()
    calls = list(_with_workspace(w).values())
    want = [f().clone() for f in calls]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0), (1, 1, 0)):
        for o in outs:
            o.fill_(7)
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i], want[i]) for i in order)


@gpu
def test_a_calls_status_is_its_own():
    """An error that other code left in the thread is neither taken for this call's nor cleared."""
    paths = {line.split()[-1] for line in open("/proc/self/maps") if "libamdhip64" in line}
    hip = ctypes.CDLL(paths.pop())
    w = _world()
    for name, call in _calls(w).items():
        want = [t.clone() for t in _flat(call())]
        torch.cuda.synchronize()
        hip.hipGetLastError()
        assert hip.hipSetDevice(4096) != 0
        got = _flat(call())
        left = hip.hipGetLastError()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got)), name
        assert left != 0 or "no rows" in name, name
