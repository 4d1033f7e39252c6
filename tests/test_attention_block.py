"""A block's attention half as a served model uses it (GPU): norms, the merged projection, the cache, attention, the output
projection and the next norms, over a prompt, a second chunk of it behind the cache, and single tokens.

    hs = block_norms(x, stream);  y = gemm(rotate_quant(hs))          q | k | v columns, bf16
    kv_write(y's k and v columns);  o = attn_prefill(y's columns)     f16, as the next prologue takes it
    z = gemm(rotate_quant(o));  stream', hs' = block_norms(z, stream)
    a later chunk:  kv_write, kv_read of everything, attn_prefill of the chunk's rows behind all keys
    one token:      kv_write, attn_decode

Every attention step is checked against its formula in 64 bits on what the steps before really wrote, with the tolerance of the
single operators."""
import numpy as np
import pytest
import torch

import rotated_w4a8_group_amd as pq
import synth
import test_attention as ta
import test_kv_cache as tk
import test_matvec as tm

pytestmark = pytest.mark.gpu

K, Hq, Hkv, D, PAGE = 1024, 12, 2, 64, 16
N = (Hq + 2 * Hkv) * D
I32 = torch.int32


class Half:
    def __init__(self, seed=800):
        self.qkv, self.out = tm.Layer(K, N, seed), tm.Layer(Hq * D // 128 * 128, K, seed + 1)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.w = [(1 + 0.2 * torch.randn(K, generator=g, device="cuda")).half() for _ in range(4)]
        self.rot = {}
        for name, width in (("in", K), ("out", Hq * D)):
            pl, tl, cl = synth.rotations(synth.Workload("attn", seed, 1, width, 128))
            self.rot[name] = (torch.from_numpy(np.stack([pq.build_records(p, t) for p, t in zip(pl, tl)])).cuda(), torch.from_numpy(np.stack(cl)).cuda())

    def project(self, x, stream):
        stream, hs = pq.block_norms(x, stream, self.w[0], None, self.w[1])
        y = pq.gemm(*pq.rotate_quant(hs, *self.rot["in"]), self.qkv.wpk, self.qkv.sz, N)
        q, k, v = y.split([Hq * D, Hkv * D, Hkv * D], 1)
        return stream, q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))

    def finish(self, o, stream):
        z = pq.gemm(*pq.rotate_quant(o.flatten(1), *self.rot["out"]), self.out.wpk, self.out.sz, K)
        return pq.block_norms(z, stream, self.w[2], None, self.w[3], scale=0.5)


class Cache:
    def __init__(self, B, longest, seed=1):
        self.width = -(-longest // PAGE)
        pages = B * self.width + 2
        order = torch.randperm(pages, generator=torch.Generator().manual_seed(seed))[:B * self.width]
        self.table = order.reshape(B, self.width).to(I32).cuda()
        self.codes = [torch.full((pages, Hkv, PAGE, D), 0x7F, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.scales = [torch.full((pages, Hkv, PAGE), float("nan"), device="cuda") for _ in range(2)]

    def slots(self, b, pos):
        return self.table[b].long()[pos // PAGE] * PAGE + pos % PAGE

    def write(self, k, v, slots):
        pq.kv_write(k, v, slots, *self.codes, *self.scales)


def _stored(x):
    """What the cache holds of rows [n, Hkv, D], in 64 bits."""
    codes, s = tk._codes(x.float().cpu().numpy())
    return (torch.from_numpy(codes).view(torch.float8_e4m3fn).double() * torch.from_numpy(np.ascontiguousarray(s)).double()[..., None]).cuda()


def _inputs(M, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn((M, K), generator=g, device="cuda").bfloat16(), (3 * torch.randn((M, K), generator=g, device="cuda")).half()


def test_prompt_chunk_and_tokens():
    half, lens, chunk, steps = Half(), [70, 1, 45], [20, 33, 1], 3
    B, cache = len(lens), Cache(3, 100)
    keys, values = [[] for _ in range(B)], [[] for _ in range(B)]

    # the prompts, packed, with padding rows behind them
    T = sum(lens) + 6
    x, stream = _inputs(T, 1)
    stream, q, k, v = half.project(x, stream)
    cu = ta._cu(lens)
    slots = torch.cat([cache.slots(b, torch.arange(n, device="cuda")) for b, n in enumerate(lens)] + [torch.full((6,), -1, device="cuda")])
    cache.write(k, v, slots)
    o = torch.zeros((T, Hq, D), dtype=torch.float16, device="cuda")
    pq.attn_prefill(q, k, v, cu, out=o)
    ta._check_prompts(o, q, k, v, [(n, n) for n in lens], 0, True, D ** -0.5, "prompts")
    assert not bool(o[sum(lens):].any())
    h, hs = half.finish(o, stream)
    assert bool(torch.isfinite(h[:sum(lens)].float()).all()) and bool(torch.isfinite(hs[:sum(lens)].float()).all())
    at = 0
    for b, n in enumerate(lens):
        keys[b], values[b] = k[at:at + n].clone(), v[at:at + n].clone()
        at += n

    # a second chunk of each, behind what the cache holds
    x, stream = _inputs(sum(chunk), 2)
    stream, q, k, v = half.project(x, stream)
    cache.write(k, v, torch.cat([cache.slots(b, torch.arange(lens[b], lens[b] + n, device="cuda")) for b, n in enumerate(chunk)]))
    total = [a + b for a, b in zip(lens, chunk)]
    kr, vr = pq.kv_read(*cache.codes, cache.table, ta._cu(total), sum(total), *cache.scales, dtype=torch.bfloat16)
    at = rat = 0
    for b, n in enumerate(chunk):
        keys[b], values[b] = torch.cat([keys[b], k[at:at + n]]), torch.cat([values[b], v[at:at + n]])
        for got, rows in ((kr, keys[b]), (vr, values[b])):
            assert torch.equal(got[rat:rat + total[b]], _stored(rows).float().bfloat16())
        at, rat = at + n, rat + total[b]
    o = pq.attn_prefill(q, kr, vr, ta._cu(chunk), ta._cu(total), dtype=torch.float16)
    ta._check_prompts(o, q, kr, vr, list(zip(chunk, total)), 0, True, D ** -0.5, "chunk")
    half.finish(o, stream)

    # tokens
    pos = torch.tensor(total, device="cuda")
    for step in range(steps):
        x, stream = _inputs(B, 10 + step)
        stream, q, k, v = half.project(x, stream)
        cache.write(k, v, torch.cat([cache.slots(b, pos[b:b + 1]) for b in range(B)]))
        pos += 1
        o = pq.attn_decode(q, *cache.codes, cache.table, pos.to(I32), *cache.scales, dtype=torch.float16)
        for b in range(B):
            keys[b], values[b] = torch.cat([keys[b], k[b:b + 1]]), torch.cat([values[b], v[b:b + 1]])
        rows = [[_stored(r) for r in keys], [_stored(r) for r in values]]
        ta._check_decode(o, q, rows, [len(r) for r in keys], D ** -0.5, f"token {step}")
        h, hs = half.finish(o, stream)
        assert bool(torch.isfinite(hs.float()).all())


def test_captured_token_steps():
    """One token's step captured once; replayed with the lengths and slots of every next token, beside eager steps of another cache."""
    half, B = Half(810), 4
    start = [5, 40, 1100, 17]
    caches = [Cache(B, 1200, s) for s in (1, 2)]
    g = torch.Generator(device="cuda").manual_seed(3)
    for c in caches:
        for b, n in enumerate(start):
            c.write(torch.randn((n, Hkv, D), generator=g, device="cuda").bfloat16(), torch.randn((n, Hkv, D), generator=g, device="cuda").bfloat16(), c.slots(b, torch.arange(n, device="cuda")))
    caches[1].codes, caches[1].scales, caches[1].table = [t.clone() for t in caches[0].codes], [t.clone() for t in caches[0].scales], caches[0].table.clone()
    x, stream = _inputs(B, 1)
    slots, lens = torch.full((B,), -1, device="cuda"), torch.tensor(start, dtype=I32, device="cuda")
    ws = torch.empty(pq.attn_decode_workspace_bytes(B, Hq, Hkv, D), dtype=torch.uint8, device="cuda")

    def step(cache, x, stream, slots, lens, ws=None):
        s, q, k, v = half.project(x, stream)
        cache.write(k, v, slots)
        return half.finish(pq.attn_decode(q, *cache.codes, cache.table, lens, *cache.scales, dtype=torch.float16, workspace=ws), s)
    step(caches[0], x, stream, slots, lens, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0], x, stream, slots, lens, ws)
    for i in range(20):
        new = _inputs(B, 20 + i)
        at = [torch.tensor([n + i], device="cuda") for n in start]
        x.copy_(new[0])
        stream.copy_(new[1])
        slots.copy_(torch.cat([caches[0].slots(b, at[b]) for b in range(B)]))
        lens.copy_(torch.cat(at) + 1)
        graph.replay()
        want = step(caches[1], *new, torch.cat([caches[1].slots(b, at[b]) for b in range(B)]), (torch.cat(at) + 1).to(I32))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(caches[0].codes + caches[0].scales, caches[1].codes + caches[1].scales))
