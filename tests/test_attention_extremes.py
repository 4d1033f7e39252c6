"""pq_attn_decode and pq_attn_prefill at the ends of what they take: queries that see no key beside values that are not finite, scales that
make one key all of the weight, values at the end of their type, weights far below the largest one. Against the formula in 64 bits.

The tolerances are those of test_attention, but for what each test says."""
import math

import pytest
import torch

import rotated_w4a8_group_amd as pq
import test_attention as ta

pytestmark = pytest.mark.gpu
F16, BF16, U8, I32 = torch.float16, torch.bfloat16, torch.uint8, torch.int32
E4M3 = torch.float8_e4m3fn
U = 2.0 ** -24


def _i32(*v):
    return torch.tensor(v, dtype=I32, device="cuda")


# ------------------------------------------------------------------------------------------
# (queries, keys): whole items, and items cut along the keys (few items, more than 1024 keys)
NO_KEY = [[(40, 20), (5, 3)], [(300, 200), (9, 9)], [(1300, 1200)], [(150, 100), (1500, 1480), (7, 2000)]]


@pytest.mark.parametrize("lens", NO_KEY)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16")])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_without_a_key_beside_values_that_are_not_finite(lens, D, kind, out, bad):
    """Rows that see no key are zeros whatever V holds; those that see keys but no bad value are as without it."""
    g = torch.Generator().manual_seed(D + len(lens))
    q, k, v, cu_q, cu_k = ta._prompts(g, lens, 2, 1, D, ta.TYPES[kind])
    v = v.clone()
    kat, first = 0, []
    for nq, nk in lens:       # a value that the first rows with keys see, one that they do not, and the last
        at = [x for x in (3, 17, 70, nk - 1) if x < nk]
        first.append(min(at))
        for x in at:
            v[kat + x, 0, x % D] = bad
        kat += nk
    o = pq.attn_prefill(q, k, v, cu_q, cu_k, dtype=ta.TYPES[out])
    at = kat = 0
    for (nq, nk), f in zip(lens, first):
        none = max(nq - nk, 0)
        assert bool((o[at:at + none] == 0).all()), (nq, nk)
        sane = max(0, min(nq, f - (nk - nq)))       # rows that see keys 0 .. f - 1 at most
        assert bool(torch.isfinite(o[at:at + sane]).all()) and not bool(torch.isfinite(o[at + sane:at + nq]).all(-1).any()), (nq, nk)
        for h in range(2):
            visible = torch.ones((sane, nk), dtype=torch.bool, device="cuda").tril(nk - nq)
            ref = ta._reference(q[at:at + sane, h].double(), k[kat:kat + nk, 0].double(), torch.nan_to_num(v[kat:kat + nk, 0].double(), 0, 0, 0), D ** -0.5, visible)
            ta._check(o[at:at + sane, h], ref, nk, D, q.dtype, ta._e_p(q, o), f"beside bad values, {(nq, nk)}, head {h}")
        at, kat = at + nq, kat + nk
