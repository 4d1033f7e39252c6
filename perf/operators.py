"""Cases of the operators that stand around the packed 4-bit linear layer: the rotation without
quantisation (``rotate``), products of few 16-bit rows with the packed weights (``matvec``), the
gated projection pair in one launch (``gemm_glu``) and the norms before and after a block with its
gate and residual scale (``block_norms``).

``run`` computes each in elementary torch operations, or with ``own`` through the package's calls;
``exact`` computes them from their definitions in 64 bits.

Weights are AWQ words (nibble order 0,2,4,6,1,3,5,7) with zero points and f16 scales per 128 rows;
the value of a weight is ``sc (c - 8) - fl16(sc (zp - 8))``, the package's scale/zero-point format.
"""
import math

import torch

own = False

GROUP = 128
LAYERS = 8
AWQ_ORDER = (0, 2, 4, 6, 1, 3, 5, 7)
NO_BOUNDARY = 0x7FFFFFFF
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def _pq():
    import rotated_w4a8_group_amd as pq
    return pq


# ------------------------------------------------------------------------------------------
# cases
def listed():
    return [
        # one decoded token before a gate_up projection whose weights are read with 16-bit activations
        {"name": "rotate_1", "op": "rotate", "M": 1, "K": 5120, "P": 1, "type": "f16"},
        # a ragged prompt chunk into a merged projection with three rotations
        {"name": "rotate_1021", "op": "rotate", "M": 1021, "K": 5120, "P": 3, "type": "bf16"},
        # one decoded token, gate_up
        {"name": "matvec_1", "op": "matvec", "M": 1, "K": 5120, "split": "17408", "type": "f16", "out": "f16"},
        # a small batch through the merged q, k, v projection with its three rotations
        {"name": "matvec_4_qkv", "op": "matvec", "M": 4, "K": 5120, "split": "6144,1024,1024", "type": "bf16", "out": "bf16"},
        # the largest batch, the down projection
        {"name": "matvec_16_down", "op": "matvec", "M": 16, "K": 17408, "split": "5120", "type": "bf16", "out": "bf16"},
        # the feed-forward's first half: one token, a speculated handful with a rotation for each projection, an odd
        # small prompt on a small layer, a prompt
        {"name": "glu_1", "op": "glu", "M": 1, "K": 5120, "F": 8704, "P": 1, "act": "silu", "out": "f16"},
        {"name": "glu_7_two_rotations", "op": "glu", "M": 7, "K": 5120, "F": 4352, "P": 2, "act": "silu", "out": "bf16"},
        {"name": "glu_301_small", "op": "glu", "M": 301, "K": 1024, "F": 1424, "P": 1, "act": "gelu", "out": "bf16"},
        {"name": "glu_2048", "op": "glu", "M": 2048, "K": 5120, "F": 8704, "P": 1, "act": "silu", "out": "f16"},
        # the residual stream between two blocks: one token; a narrow model with a 32-bit stream, a gate row for
        # every token; a long prompt with channel gates
        {"name": "norms_1", "op": "norms", "M": 1, "K": 5120, "x": "bf16", "res": "f16", "out": "f16", "post": True,
         "gate": "none", "gate_act": "none", "scale": 1.0, "res_scale": 1.0, "gemma": True},
        {"name": "norms_333_narrow", "op": "norms", "M": 333, "K": 1000, "x": "bf16", "res": "f32", "out": "bf16", "post": True,
         "gate": "rows", "gate_act": "sigmoid", "scale": 0.22, "res_scale": 1.0, "gemma": False},
        {"name": "norms_8192", "op": "norms", "M": 8192, "K": 5120, "x": "bf16", "res": "f16", "out": "f16", "post": True,
         "gate": "channel", "gate_act": "none", "scale": 1.0, "res_scale": 0.5, "gemma": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotate", "matvec", "glu", "norms"))
    if op == "rotate":
        P, K = rng.randint(1, 3), GROUP * _log(rng, 1, 136)
        return {"op": op, "M": _log(rng, 1, max(2, min(4096, 1021 * 5120 * 3 // (K * P)))), "K": K, "P": P,
                "type": rng.choice(("f16", "bf16"))}
    if op == "matvec":
        P, K = rng.randint(1, 3), GROUP * _log(rng, 1, 136)
        most = 5120 * 17408 // K
        widths = [GROUP * _log(rng, 1, max(1, min(136, most // GROUP // P))) for _ in range(P)]
        widths[-1] += 16 * rng.randint(0, 7)      # the last partition may end on any 16-column line
        return {"op": op, "M": rng.randint(1, 16), "K": K, "split": ",".join(map(str, widths)),
                "type": rng.choice(("f16", "bf16")), "out": rng.choice(("f16", "bf16"))}
    if op == "glu":
        K, F = GROUP * _log(rng, 1, 80), 16 * _log(rng, 1, 544)
        M = rng.choice((_log(rng, 1, 16), _log(rng, 17, max(18, min(2048, 2048 * 5120 * 8704 // (K * F))))))
        return {"op": op, "M": M, "K": K, "F": F, "P": rng.choice((1, 1, 2)) if F % GROUP == 0 else 1,
                "act": rng.choice(("silu", "gelu")), "out": rng.choice(("f16", "bf16"))}
    K = 8 * _log(rng, 1, 2304)
    return {"op": op, "M": _log(rng, 1, max(2, min(16384, 8192 * 5120 // K // 2))), "K": K, "x": rng.choice(("f16", "bf16")),
            "res": rng.choice(("f16", "bf16", "f32")), "out": rng.choice(("f16", "bf16")), "post": rng.random() < 0.7,
            "gate": rng.choice(("none", "channel", "token", "rows")), "gate_act": rng.choice(("none", "sigmoid", "tanh")),
            "scale": rng.choice((1.0, 0.22)), "res_scale": rng.choice((1.0, 0.5)), "gemma": rng.random() < 0.5}


# ------------------------------------------------------------------------------------------
# inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _awq(codes):
    """Codes 0..15 [R, N] -> int32 words [R, N/8]."""
    words = torch.zeros((codes.shape[0], codes.shape[1] // 8), dtype=torch.int32, device="cuda")
    for i, column in enumerate(AWQ_ORDER):
        words |= codes[:, column::8].to(torch.int32) << (4 * i)
    return words


def _weights(g, K, N):
    s = {"qweight": _awq(torch.randint(0, 16, (K, N), generator=g, device="cuda", dtype=torch.uint8)),
         "qzeros": _awq(torch.randint(2, 15, (K // GROUP, N), generator=g, device="cuda", dtype=torch.uint8)),
         "scales": (0.002 + 0.018 * torch.rand((K // GROUP, N), generator=g, device="cuda")).half()}
    if own:   # laid out once, when the layer is loaded
        s["wpk"], s["sz"] = _pq().pack_weights(s["qweight"], s["qzeros"], s["scales"])
    return s


def _rows(g, shape):
    """Activations: each token with a size of its own, one channel in a hundred 20 times as large."""
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp(0.5 * torch.randn(shape[:-1] + (1,), generator=g, device="cuda"))
    return x * torch.where(torch.rand(shape[-1], generator=g, device="cuda") < 0.01, 20.0, 1.0)


def prepare(case, seed):
    g, op, M, K = _gen(seed), case["op"], case["M"], case["K"]
    s = dict(case)
    if op == "rotate":
        P, G = case["P"], K // GROUP
        s["x"] = _rows(g, (M, K)).to(TYPES[case["type"]])
        pairs = torch.rand((P, LAYERS, G, GROUP), generator=g, device="cuda").argsort(-1)
        theta = ((2 * torch.rand((P, LAYERS, K // 2), generator=g, device="cuda") - 1) * math.pi).half()
        s["cs"] = torch.exp(0.3 * torch.randn((P, K), generator=g, device="cuda")).half()
        # the pairs' channels and the f16 cosines and sines: the plan that a program makes at load
        at = (pairs + GROUP * torch.arange(G, device="cuda")[:, None]).reshape(P, LAYERS, K // 2, 2)
        s["first"], s["second"] = at[..., 0].contiguous(), at[..., 1].contiguous()
        s["cos"], s["sin"] = torch.cos(theta.double()).half(), torch.sin(theta.double()).half()
        if own:
            pq = _pq()
            pn, tn = pairs.reshape(P, LAYERS, K).short().cpu().numpy(), theta.cpu().numpy()
            s["rec"] = torch.stack([torch.from_numpy(pq.build_records(pn[p], tn[p])) for p in range(P)]).cuda()
            s["y"] = torch.empty((P, M, K), dtype=s["x"].dtype, device="cuda")
    elif op == "matvec":
        widths = [int(w) for w in case["split"].split(",")]
        ends = [sum(widths[:i + 1]) for i in range(len(widths))]
        s["N"], s["ends"] = ends[-1], ends
        s["pb"] = (ends[:-1] + [NO_BOUNDARY] * 2)[:2]
        s["x"] = _rows(g, (len(widths), M, K)).to(TYPES[case["type"]])
        s.update(_weights(g, K, s["N"]))
        if own:
            s["y"] = torch.empty((M, s["N"]), dtype=TYPES[case["out"]], device="cuda")
    elif op == "glu":
        P, F = case["P"], case["F"]
        v = _rows(g, (P, M, K // GROUP, GROUP))
        s["ASG"] = v.abs().amax(-1) / 448
        s["A"] = (v / s["ASG"][..., None]).to(torch.float8_e4m3fn)
        s["RS"] = s["A"].float().sum(-1)
        s["A"] = s["A"].view(torch.uint8).reshape(P, M, K)
        s.update(_weights(g, K, 2 * F))
        if own:
            pq = _pq()
            s["h"] = torch.empty((M, F), dtype=TYPES[case["out"]], device="cuda")
            n = pq.gemm_workspace_bytes(M, 2 * F, K)
            s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    else:
        s["eps"] = 1e-6
        s["x"] = (2 * _rows(g, (M, K))).to(TYPES[case["x"]])
        s["res"] = (4 * _rows(g, (M, K))).to(TYPES[case["res"]])
        w = 0.3 * torch.randn((2, K), generator=g, device="cuda") + (0.0 if case["gemma"] else 1.0)
        w = w.to(TYPES[case["out"]])
        s["w_post"], s["w_pre"] = (w[0].contiguous() if case["post"] else None), w[1].contiguous()
        shape = {"none": None, "channel": (K,), "token": (M, 1), "rows": (M, K)}[case["gate"]]
        s["gate"] = None if shape is None else torch.randn(shape, generator=g, device="cuda").to(TYPES[case["x"]])
        if own:
            s["h"], s["hs"] = torch.empty_like(s["res"]), torch.empty((M, K), dtype=TYPES[case["out"]], device="cuda")
    return s


# ------------------------------------------------------------------------------------------
# the package's calls
def _run_own(s):
    pq, op = _pq(), s["op"]
    if op == "rotate":
        return pq.rotate(s["x"], s["rec"], s["cs"], out=s["y"])
    if op == "matvec":
        return pq.matvec(s["x"], s["wpk"], s["sz"], s["N"], s["pb"][0], s["pb"][1], out=s["y"])
    if op == "glu":
        return pq.gemm_glu(s["A"], s["ASG"], s["RS"], s["wpk"], s["sz"], s["F"], act=s["act"], out=s["h"], workspace=s["ws"])
    return pq.block_norms(s["x"], s["res"], w_post=s["w_post"], gate=s["gate"], w_pre=s["w_pre"], eps=s["eps"],
                          scale=s["scale"], res_scale=s["res_scale"], gate_act=s["gate_act"], gemma=s["gemma"],
                          residual_out=s["h"], out=s["hs"])


# ------------------------------------------------------------------------------------------
# plain forms
def _unpack(words):
    """AWQ words [R, N/8] -> codes [R, N]."""
    shift = torch.tensor([4 * AWQ_ORDER.index(c) for c in range(8)], dtype=torch.int32, device=words.device)
    return ((words[..., None] >> shift) & 15).reshape(words.shape[0], -1)


def _dequant(s):
    K = s["qweight"].shape[0]
    sc = s["scales"].float()
    zsc = (sc * (_unpack(s["qzeros"]) - 8)).half().float()
    w = (_unpack(s["qweight"]) - 8).float().reshape(K // GROUP, GROUP, -1)
    return (w * sc[:, None] - zsc[:, None]).reshape(K, -1)


def _plain_rotate(s):
    out = []
    for p in range(s["P"]):
        v = s["x"].float() * s["cs"][p].float()
        for r in range(LAYERS):
            i, j, c, n = s["first"][p, r], s["second"][p, r], s["cos"][p, r].float(), s["sin"][p, r].float()
            a, b = v[:, i], v[:, j]
            v = torch.empty_like(v)
            v[:, i], v[:, j] = c * a + n * b, c * b - n * a
        out.append(v.to(s["x"].dtype))
    return torch.stack(out)


def _plain_matvec(s):
    w, x = _dequant(s), s["x"].float()
    begins = [0] + s["ends"][:-1]
    return torch.cat([x[p] @ w[:, a:b] for p, (a, b) in enumerate(zip(begins, s["ends"]))], 1).to(TYPES[s["out"]])


def _plain_glu(s):
    F, (P, M, K) = s["F"], s["A"].shape
    a = s["A"].view(torch.float8_e4m3fn).float().reshape(P, M, K // GROUP, GROUP)
    a = (a * s["ASG"][..., None]).reshape(P, M, K)
    w = _dequant(s)
    g, u = a[0] @ w[:, :F], a[P - 1] @ w[:, F:]
    if s["act"] == "silu":
        g = g / (1 + torch.exp(-g))
    else:
        g = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))
    return (g * u).to(TYPES[s["out"]])


def _plain_norms(s):
    one = 1.0 if s["gemma"] else 0.0
    n = s["x"].float()
    if s["w_post"] is not None:
        n = n * torch.rsqrt((n * n).mean(-1, keepdim=True) + s["eps"]) * (one + s["w_post"].float())
    if s["gate"] is not None:
        t = s["gate"].float()
        t = 1 / (1 + torch.exp(-t)) if s["gate_act"] == "sigmoid" else torch.tanh(t) if s["gate_act"] == "tanh" else t
        n = n * t
    h = (s["res_scale"] * s["res"].float() + s["scale"] * n).to(s["res"].dtype)
    f = h.float()
    hs = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + s["eps"]) * (one + s["w_pre"].float())
    return h, hs.to(TYPES[s["out"]])


def run(state):
    if own:
        return _run_own(state)
    return {"rotate": _plain_rotate, "matvec": _plain_matvec, "glu": _plain_glu, "norms": _plain_norms}[state["op"]](state)


# ------------------------------------------------------------------------------------------
# what a pass cannot do without
def work(case):
    op, M, K = case["op"], case["M"], case["K"]
    G = K // GROUP
    if op == "rotate":
        P = case["P"]
        return {"bytes": 2 * M * K * (1 + P) + P * (8 * LAYERS * K // 2 + 2 * K), "flops": M * P * (K + 6 * LAYERS * K // 2)}
    if op == "matvec":
        widths = [int(w) for w in case["split"].split(",")]
        N = sum(widths)
        return {"bytes": K * N // 2 + 4 * G * N + 2 * len(widths) * M * K + 2 * M * N, "flops": 2 * M * N * K}
    if op == "glu":
        P, F = case["P"], case["F"]
        return {"bytes": K * F + 8 * G * F + P * M * (K + 8 * G) + 2 * M * F, "flops": 4 * M * F * K}
    size = {"f16": 2, "bf16": 2, "f32": 4}
    gate = {"none": 0, "channel": K, "token": M, "rows": M * K}[case["gate"]]
    return {"bytes": M * K * (size[case["x"]] + 2 * size[case["res"]] + size[case["out"]]) + 2 * gate +
            2 * K * (1 + case["post"]), "flops": M * K * (10 if case["post"] else 6)}


# ------------------------------------------------------------------------------------------
# the definitions in 64 bits
def _exact_product(x, s, first, last):
    """x (64 bits) times the weights' columns first..last-1, one nibble position of the words at a time."""
    K = x.shape[1]
    y = torch.empty((x.shape[0], last - first), dtype=torch.float64, device=x.device)
    words, zeros = s["qweight"][:, first // 8:last // 8], s["qzeros"][:, first // 8:last // 8]
    for i, column in enumerate(AWQ_ORDER):
        sc = s["scales"][:, first:last][:, column::8].double()
        zsc = (sc * (((zeros >> (4 * i)) & 15).double() - 8)).half().double()
        c = ((words >> (4 * i)) & 15).double()
        w = torch.repeat_interleave(sc, GROUP, 0) * (c - 8) - torch.repeat_interleave(zsc, GROUP, 0)
        y[:, column::8] = x @ w
    return y


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rotate":
        M, K, P = case["M"], case["K"], case["P"]
        G, out = K // GROUP, []
        for p in range(P):
            # every group's eight layers as one 128 x 128 matrix: a layer is cos on the diagonal, and +-sin where the pairs meet
            m = torch.eye(GROUP, dtype=torch.float64, device="cuda").repeat(G, 1, 1)
            for r in range(LAYERS):
                i, j = s["first"][p, r].reshape(G, -1) % GROUP, s["second"][p, r].reshape(G, -1) % GROUP
                c, n = s["cos"][p, r].double().reshape(G, -1), s["sin"][p, r].double().reshape(G, -1)
                layer = torch.zeros_like(m)
                k = torch.arange(G, device="cuda")[:, None]
                layer[k, i, i], layer[k, j, j], layer[k, j, i], layer[k, i, j] = c, c, n, -n
                m = torch.bmm(m, layer)
            v = (s["x"].double() * s["cs"][p].double()).reshape(M, G, GROUP).transpose(0, 1).contiguous()
            out.append(torch.bmm(v, m).transpose(0, 1).reshape(M, K))
        return torch.stack(out)
    if op == "matvec":
        begins = [0] + s["ends"][:-1]
        return torch.cat([_exact_product(s["x"][p].double(), s, a, b) for p, (a, b) in enumerate(zip(begins, s["ends"]))], 1)
    if op == "glu":
        F, x = s["F"], s["A"].view(torch.float8_e4m3fn).double() * torch.repeat_interleave(s["ASG"].double(), GROUP, -1)
        g, u = _exact_product(x[0], s, 0, F), _exact_product(x[-1], s, F, 2 * F)
        if case["act"] == "silu":
            return g * torch.sigmoid(g) * u
        return g * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)) * u
    x, res, one = s["x"].double(), s["res"].double(), 1.0 if case["gemma"] else 0.0
    if case["post"]:
        x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / case["K"] + s["eps"]) * (s["w_post"].double() + one)
    if s["gate"] is not None:
        t = s["gate"].double()
        x = x * {"none": t, "sigmoid": torch.sigmoid(t), "tanh": torch.tanh(t)}[case["gate_act"]]
    h = case["res_scale"] * res + case["scale"] * x
    r = h.to(s["res"].dtype).double()
    return h, r / torch.sqrt(r.square().sum(-1, keepdim=True) / case["K"] + s["eps"]) * (s["w_pre"].double() + one)
