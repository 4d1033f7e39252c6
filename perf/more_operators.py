"""Cases of the key-value cache and the attention that reads it: rows quantised as they are written into a
paged cache (``kv_write``) and read back (``kv_read``), attention of one new token of each sequence over that
cache (``attn_decode``) and causal attention over packed prompts with grouped heads (``attn_prefill``).

``run`` computes each in elementary torch operations, or with ``own`` through the package's calls;
``exact`` computes them from their definitions in 64 bits.

A cache holds [pages, kv heads, rows of a page, head size]: e4m3 codes with a binary32 scale for each (row, head),
max |x| / 448, or the 16-bit values themselves. Query i of a sequence of nq queries and nk keys sees the keys
j <= i + nk - nq; a query that sees no key gives zeros.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8}
E4M3 = torch.float8_e4m3fn


def _pq():
    import rotated_w4a8_group_amd as pq
    return pq


# ------------------------------------------------------------------------------------------
# cases
def listed():
    return [
        # the cache's side of one decoded token: the k and v columns of one row of the merged projection
        {"name": "write_1", "op": "write", "T": 1, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16", "cache": "e4m3", "page": 16, "padding": 0},
        # a prompt chunk with padding rows behind it
        {"name": "write_4099", "op": "write", "T": 4099, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16", "cache": "e4m3", "page": 16, "padding": 61},
        # the rows of one short sequence read back, as the next chunk of its prompt needs them
        {"name": "read_65", "op": "read", "B": 1, "longest": 65, "lengths": 0, "Hkv": 4, "D": 256, "cache": "e4m3", "out": "f16", "page": 64},
        # those of a batch of long ones
        {"name": "read_ragged", "op": "read", "B": 7, "longest": 8191, "lengths": 5, "Hkv": 8, "D": 128, "cache": "e4m3", "out": "bf16", "page": 16},
        # one decoded token: a chat's first answer, a very long document; a small batch with wide heads; a full batch of
        # ragged lengths with a 16-bit cache
        {"name": "decode_1_short", "op": "decode", "B": 1, "longest": 509, "lengths": 0, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16",
         "cache": "e4m3", "out": "f16", "page": 16},
        {"name": "decode_1_long", "op": "decode", "B": 1, "longest": 131071, "lengths": 0, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16",
         "cache": "e4m3", "out": "f16", "page": 64},
        {"name": "decode_17_wide", "op": "decode", "B": 17, "longest": 4000, "lengths": 7, "Hq": 24, "Hkv": 4, "D": 256, "type": "f16",
         "cache": "e4m3", "out": "f16", "page": 16},
        {"name": "decode_64_ragged", "op": "decode", "B": 64, "longest": 8192, "lengths": 3, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16",
         "cache": "bf16", "out": "bf16", "page": 32},
        # prompts: one short question; a packed batch of ragged ones; a chunk of a long prompt behind the rows read back
        # from the cache, with wide heads; one long prompt
        {"name": "prefill_37", "op": "prefill", "B": 1, "T": 37, "lengths": 0, "prefix": 0, "Hq": 12, "Hkv": 12, "D": 64, "type": "f16", "out": "f16"},
        {"name": "prefill_packed", "op": "prefill", "B": 9, "T": 4093, "lengths": 11, "prefix": 0, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16",
         "out": "bf16"},
        {"name": "prefill_chunk_wide", "op": "prefill", "B": 1, "T": 512, "lengths": 0, "prefix": 8191, "Hq": 24, "Hkv": 4, "D": 256, "type": "bf16",
         "out": "bf16"},
        {"name": "prefill_8192", "op": "prefill", "B": 1, "T": 8192, "lengths": 0, "prefix": 0, "Hq": 48, "Hkv": 8, "D": 128, "type": "bf16",
         "out": "bf16"},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    D = rng.choice((64, 128, 256))
    return D, _log(rng, 1, 16 if D < 256 else 8), rng.choice((1, 1, 2, 4, 5, 6, 7, 8, 16))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "prefill"))
    D, Hkv, G = _heads(rng)
    page, lengths = 16 << rng.randint(0, 4), rng.randint(1, 10 ** 6)
    if op == "write":
        T = _log(rng, 1, 4099 * 8 * 128 // (Hkv * D))
        t = rng.choice(("f16", "bf16"))
        return {"op": op, "T": T, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "type": t, "cache": rng.choice(("e4m3", "e4m3", t)), "page": page,
                "padding": rng.choice((0, T // 7))}
    if op == "read":
        B = _log(rng, 1, 64)
        t = rng.choice(("f16", "bf16"))
        return {"op": op, "B": B, "longest": _log(rng, 1, max(2, min(65536, 25000 * 8 * 128 // (B * Hkv * D)))), "lengths": lengths, "Hkv": Hkv, "D": D,
                "cache": rng.choice(("e4m3", "e4m3", t)), "out": t, "page": page}
    if op == "decode":
        B = _log(rng, 1, 128)
        t = rng.choice(("f16", "bf16"))
        return {"op": op, "B": B, "longest": _log(rng, 1, max(2, min(131072, 160000 * 8 * 128 // (B * Hkv * D)))), "lengths": lengths, "Hq": G * Hkv,
                "Hkv": Hkv, "D": D, "type": t, "cache": rng.choice(("e4m3", "e4m3", t)), "out": rng.choice(("f16", "bf16")), "page": page}
    Hkv = min(Hkv, max(1, 48 // G))
    prefix = rng.choice((0, 0, 0, _log(rng, 1, 8192)))
    T = _log(rng, 1, 8192)
    while T * (T + 12 * prefix) * G * Hkv * D > 8192 * 8192 * 48 * 128:
        T = T * 3 // 4
    B = min(T, _log(rng, 1, 12))
    t = rng.choice(("f16", "bf16"))
    return {"op": op, "B": B, "T": T, "lengths": lengths, "prefix": prefix, "Hq": G * Hkv, "Hkv": Hkv, "D": D, "type": t,
            "out": rng.choice((t, t, "f16", "bf16"))}


def _lengths(case):
    """Lengths of the cached sequences: the longest, and others spread below it, empty ones among them."""
    r = random.Random(case["lengths"])
    return [case["longest"]] + [int((case["longest"] + 1) * r.random() ** 1.5) for _ in range(case["B"] - 1)]


def _prompts(case):
    """Lengths of the packed prompts, T rows in all."""
    r = random.Random(case["lengths"])
    cuts = sorted(int(case["T"] * r.random() ** 2) for _ in range(case["B"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["T"]])]


# ------------------------------------------------------------------------------------------
# inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(g, T, H, D):
    """Head rows: each with a size of its own, one channel in sixteen 4 times as large."""
    x = torch.randn((T, H, D), generator=g, device="cuda")
    x *= torch.exp(0.3 * torch.randn((T, H, 1), generator=g, device="cuda"))
    return x * torch.where(torch.rand((H, D), generator=g, device="cuda") < 1 / 16, 4.0, 1.0)


def _merged(g, T, Hq, Hkv, D, dtype):
    """The merged projection's rows, and their q, k and v columns as heads."""
    y = torch.cat([0.7 * _rows(g, T, Hq, D), _rows(g, T, 2 * Hkv, D)], 1).to(dtype).reshape(T, -1)
    q, k, v = y.split([Hq * D, Hkv * D, Hkv * D], 1)
    return q.unflatten(1, (Hq, D)), k.unflatten(1, (Hkv, D)), v.unflatten(1, (Hkv, D))


def _cu(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def _cache(g, pages, Hkv, page, D, kind, s):
    """A filled cache: rows of a finished prompt, and whatever the last pages still hold behind them."""
    for name in ("k", "v"):
        x = _rows(g, pages * page, Hkv, D).reshape(pages, page, Hkv, D).transpose(1, 2)
        if kind == "e4m3":
            scale = x.abs().amax(-1) / 448
            s[name + "_scale"] = scale.contiguous()
            s[name + "_cache"] = (x / scale[..., None]).to(E4M3).view(torch.uint8).contiguous()
        else:
            s[name + "_scale"] = None
            s[name + "_cache"] = x.to(TYPES[kind]).contiguous()


def prepare(case, seed):
    g, op, D = _gen(seed), case["op"], case["D"]
    s = dict(case)
    if op == "write":
        T, Hkv, page = case["T"], case["Hkv"], case["page"]
        _, s["k"], s["v"] = _merged(g, T, case["Hq"], Hkv, D, TYPES[case["type"]])
        live = T - case["padding"]
        pages = -(-live // page) + 3
        order = torch.randperm(pages, generator=g, device="cuda")
        at = torch.arange(live, device="cuda") + page // 3       # the sequence goes on inside a page
        s["slots"] = torch.cat([order[at // page] * page + at % page, torch.full((T - live,), -1, device="cuda")])
        for name in ("k", "v"):                                  # what the pages held before
            if case["cache"] == "e4m3":
                s[name + "_cache"] = torch.randint(0, 0x7F, (pages, Hkv, page, D), generator=g, device="cuda", dtype=torch.uint8)
                s[name + "_scale"] = torch.rand((pages, Hkv, page), generator=g, device="cuda")
            else:
                s[name + "_cache"] = torch.randn((pages, Hkv, page, D), generator=g, device="cuda").to(TYPES[case["cache"]])
                s[name + "_scale"] = None
    elif op in ("read", "decode"):
        lens, page, Hkv = _lengths(case), case["page"], case["Hkv"]
        need = [-(-n // page) for n in lens]
        width = max(1, max(need))
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        _cache(g, pages, Hkv, page, D, case["cache"], s)
        table = torch.full((case["B"], width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        s["table"] = table
        if op == "read":
            s["T"], s["cu"] = sum(lens), _cu(lens)
            if own:
                s["out_rows"] = tuple(torch.empty((s["T"], Hkv, D), dtype=TYPES[case["out"]], device="cuda") for _ in range(2))
        else:
            s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
            s["q"] = (0.7 * _rows(g, case["B"], case["Hq"], D)).to(TYPES[case["type"]])
            if own:
                n = _pq().attn_decode_workspace_bytes(case["B"], case["Hq"], Hkv, D)
                s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
                s["o"] = torch.empty((case["B"], case["Hq"], D), dtype=TYPES[case["out"]], device="cuda")
    else:
        lens, T, Hq, Hkv = _prompts(case), case["T"], case["Hq"], case["Hkv"]
        s["q"], s["k"], s["v"] = _merged(g, T, Hq, Hkv, D, TYPES[case["type"]])
        s["cu_q"] = s["cu_k"] = _cu(lens)
        if case["prefix"]:                                       # keys and values read back in front of each chunk's own
            Tk = T + case["prefix"] * case["B"]
            s["k"], s["v"] = (_rows(g, Tk, Hkv, D).to(TYPES[case["type"]]) for _ in range(2))
            s["cu_k"] = _cu([n + case["prefix"] for n in lens])
        if own:
            n = _pq().attn_prefill_workspace_bytes(case["B"], T, s["k"].shape[0], Hq, Hkv, D)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
            s["o"] = torch.empty((T, Hq, D), dtype=TYPES[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# the package's calls
def _as_values(s):
    """The written caches; codes as the values they stand for, beside their scales."""
    if s["k_scale"] is None:
        return s["k_cache"], s["v_cache"]
    return s["k_cache"].view(E4M3), s["v_cache"].view(E4M3), s["k_scale"], s["v_scale"]


def _run_own(s):
    pq, op = _pq(), s["op"]
    if op == "write":
        pq.kv_write(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"])
        return _as_values(s)
    if op == "read":
        return pq.kv_read(s["k_cache"], s["v_cache"], s["table"], s["cu"], s["T"], s["k_scale"], s["v_scale"], out=s["out_rows"])
    if op == "decode":
        return pq.attn_decode(s["q"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["k_scale"], s["v_scale"], out=s["o"], workspace=s["ws"])
    return pq.attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["o"], workspace=s["ws"])


# ------------------------------------------------------------------------------------------
# plain forms
def _plain_write(s):
    page = s["page"]
    keep = (s["slots"] >= 0).nonzero()[:, 0]
    slot = s["slots"][keep]
    p, r = slot // page, slot % page
    for name in ("k", "v"):
        x = s[name][keep]
        if s["k_scale"] is None:
            s[name + "_cache"][p, :, r] = x
        else:
            x = x.float()
            scale = x.abs().amax(-1) * (1 / 448)
            inverse = torch.where(scale > 0, 1 / scale, 0)
            s[name + "_cache"][p, :, r] = (x * inverse[..., None]).to(E4M3).view(torch.uint8)
            s[name + "_scale"][p, :, r] = scale
    return _as_values(s)


def _cached(s, name):
    """The cached rows of every sequence, padded to the table's width, [B, Hkv, L, D] in 32 bits."""
    table = s["table"].clamp(min=0).long()
    x = s[name + "_cache"][table]
    if s[name + "_scale"] is None:
        x = x.float()
    else:
        x = x.view(E4M3).float() * s[name + "_scale"][table][..., None]
    return x.transpose(1, 2).flatten(2, 3)


def _plain_read(s):
    pos = torch.arange(s["T"], device="cuda")
    b = (pos[:, None] >= s["cu"][1:]).sum(-1)
    at = pos - s["cu"][b]
    return tuple(_cached(s, name)[b, :, at].to(TYPES[s["out"]]) for name in ("k", "v"))


def _plain_decode(s):
    B, Hq, D = s["q"].shape
    k, v = _cached(s, "k"), _cached(s, "v")
    a = torch.matmul(s["q"].float().reshape(B, s["Hkv"], -1, D), k.transpose(2, 3)) * D ** -0.5
    seen = torch.arange(k.shape[2], device="cuda") < s["lens"][:, None]
    a = a.masked_fill(~seen[:, None, None], -math.inf)
    m = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(m == -math.inf, 0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(total > 0, total, 1)
    return o.reshape(B, Hq, D).to(TYPES[s["out"]])


def _plain_prefill(s):
    T, Hq, D = s["q"].shape
    Tk, Hkv = s["k"].shape[:2]
    iq, ik = torch.arange(T, device="cuda"), torch.arange(Tk, device="cuda")
    bq, bk = (iq[:, None] >= s["cu_q"][1:]).sum(-1), (ik[:, None] >= s["cu_k"][1:]).sum(-1)
    last = iq - s["cu_q"][bq + 1] + s["cu_k"][bq + 1]           # the last key's row that each query sees
    seen = (bq[:, None] == bk) & (ik <= last[:, None])
    q = s["q"].float().reshape(T, Hkv, -1, D).permute(1, 2, 0, 3).reshape(Hkv, -1, D)
    k, v = (s[name].float().transpose(0, 1).contiguous() for name in ("k", "v"))
    a = torch.matmul(q, k.transpose(1, 2).contiguous()).reshape(Hkv, -1, T, Tk) * D ** -0.5
    a = a.masked_fill(~seen, -math.inf)
    m = a.amax(-1, keepdim=True)
    p = torch.exp(a - torch.where(m == -math.inf, 0, m))
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(Hkv, -1, Tk), v).reshape(Hkv, -1, T, D) / torch.where(total > 0, total, 1)
    return o.permute(2, 0, 1, 3).reshape(T, Hq, D).to(TYPES[s["out"]])


def run(state):
    if own:
        return _run_own(state)
    return {"write": _plain_write, "read": _plain_read, "decode": _plain_decode, "prefill": _plain_prefill}[state["op"]](state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
def work(case):
    op, D = case["op"], case["D"]
    if op == "prefill":
        pairs = sum(n * (n + 1) // 2 + n * case["prefix"] for n in _prompts(case))
        T, Tk = case["T"], case["T"] + case["prefix"] * case["B"]
        return {"bytes": 4 * T * case["Hq"] * D + 4 * Tk * case["Hkv"] * D, "flops": 4 * pairs * case["Hq"] * D}
    row = 2 * case["Hkv"] * (D + 4 if case["cache"] == "e4m3" else 2 * D)   # bytes of a cached row, k and v
    if op == "write":
        n = case["T"] - case["padding"]
        return {"bytes": n * (4 * case["Hkv"] * D + row) + 8 * case["T"], "flops": 6 * n * case["Hkv"] * D}
    lens = _lengths(case)
    table = 4 * sum(-(-n // case["page"]) for n in lens)
    if op == "read":
        return {"bytes": sum(lens) * (row + 4 * case["Hkv"] * D) + table, "flops": 2 * sum(lens) * case["Hkv"] * D}
    return {"bytes": sum(lens) * row + 4 * case["B"] * case["Hq"] * D + table, "flops": 4 * sum(lens) * case["Hq"] * D}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
def _nearest_e4m3(x):
    """The e4m3 values nearest to x, of two equally near the one with the even code."""
    codes = torch.arange(127, device="cuda")
    exponent, fraction = codes // 8, (codes % 8).double()
    values = torch.where(exponent == 0, fraction * 2.0 ** -9, (8 + fraction) * torch.exp2((exponent - 10).double()))
    middle = (values[1:] + values[:-1]) / 2
    low = torch.bucketize(x.abs(), middle)                       # a middle itself counts as below it
    tie = (low < 126) & (x.abs() == middle[low.clamp(max=125)]) & (low % 2 == 1)
    return torch.copysign(values[low + tie.long()], x)


def _sequence(s, b, n, name):
    """The n cached rows of sequence b in 64 bits, [Hkv, n, D]."""
    used = s["table"][b, :-(-n // s["page"])].long()
    x = s[name + "_cache"][used]
    x = x.double() if s[name + "_scale"] is None else x.view(E4M3).double() * s[name + "_scale"][used].double().unsqueeze(-1)
    return torch.cat(list(x), 1)[:, :n] if len(used) else x.new_zeros((s["Hkv"], 0, s["D"]))


def _softmax_rows(q, k, v, hidden=None):
    """q [R, D], k and v [n, D] in 64 bits."""
    if k.shape[0] == 0:
        return torch.zeros_like(q)
    a = (q @ k.t().contiguous()) / math.sqrt(q.shape[1])
    if hidden is not None:
        a[hidden] = -math.inf
    return torch.nan_to_num(torch.softmax(a, -1)) @ v


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "write":
        live = case["T"] - case["padding"]
        out, scales = [], []
        for name in ("k", "v"):
            cache, scale = s[name + "_cache"], s[name + "_scale"]
            cache = (cache.view(E4M3) if scale is not None else cache).double()
            scale = None if scale is None else scale.double()
            x, slot = s[name][:live].double(), s["slots"][:live]
            for h in range(case["Hkv"]):
                rows = x[:, h]
                if scale is not None:
                    most = rows.abs().amax(-1) / 448
                    scale[slot // case["page"], h, slot % case["page"]] = most
                    rows = _nearest_e4m3(rows / torch.where(most > 0, most, 1)[:, None])
                cache[slot // case["page"], h, slot % case["page"]] = rows
            out.append(cache)
            scales.append(scale)
        return (*out, *scales) if scales[0] is not None else tuple(out)
    if op == "read":
        return tuple(torch.cat([_sequence(s, b, n, name).transpose(0, 1) for b, n in enumerate(_lengths(case))]) for name in ("k", "v"))
    G = case["Hq"] // case["Hkv"]
    if op == "decode":
        o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(_lengths(case)):
            k, v = _sequence(s, b, n, "k"), _sequence(s, b, n, "v")
            for h in range(case["Hkv"]):
                o[b, h * G:(h + 1) * G] = _softmax_rows(s["q"][b, h * G:(h + 1) * G].double(), k[h], v[h])
        return o
    o = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at, kat = 0, 0
    for n in _prompts(case):
        nk = n + case["prefix"]
        hidden = torch.ones((n, nk), dtype=torch.bool, device="cuda").triu(nk - n + 1)
        for h in range(case["Hq"]):
            k, v = (s[name][kat:kat + nk, h // G].double() for name in ("k", "v"))
            o[at:at + n, h] = _softmax_rows(s["q"][at:at + n, h].double(), k, v, hidden)
        at, kat = at + n, kat + nk
    return o
