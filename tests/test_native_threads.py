"""Calls from two Python threads at once, each on a stream and with a workspace of its own, gemm_glu's two-kernel form among them (GPU)."""
import threading
import traceback

import pytest
import torch

import rotated_w4a8_group_amd as pq
import test_gemm_glu as tg
import test_native_calls as tn

ROUNDS = 20


def _run_in_threads(n, work):
    """work(i) in n threads; what any of them raises, as text."""
    failed, done = [], [0] * n

    def guarded(i):
        try:
            for _ in work(i):
                done[i] += 1
        except BaseException:   # noqa: B902  a thread's exception ends nothing by itself
            failed.append(traceback.format_exc())
    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    return failed, done


def test_what_a_thread_raises_is_seen():
    def work(i):
        yield
        if i:
            raise ValueError("seen")
        yield
    failed, done = _run_in_threads(2, work)
    assert len(failed) == 1 and "seen" in failed[0] and done == [2, 1]


@pytest.mark.gpu
@pytest.mark.parametrize("native", [True, False])
def test_two_threads(native):
    """Through the compiled calls and, with those switched off, through Python and ctypes."""
    flat = lambda r: [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]   # noqa: E731
    pair, two = tg.Pair(256, 4640, 900), tg.Pair(640, 8704, 901)
    calls = []
    for i in range(2):
        w = tn._world()
        own = [c for n, c in tn._calls(w).items()]
        for M, p, P in ((1300, pair, 1), (700, two, 2)):      # past the row blocks: a pass writes the workspace, the tiles read it
            codes = tg._codes(P, M, p.K, 910 + 10 * i + P)
            ws = torch.empty(pq.gemm_workspace_bytes(M, 2 * p.F, p.K), dtype=torch.uint8, device="cuda")
            own += [lambda c=codes, p=p, ws=ws: pq.gemm_glu(*c, p.wpk, p.sz, p.F, workspace=ws), lambda c=codes, p=p: pq.gemm_glu(*c, p.wpk, p.sz, p.F)]
        calls.append(own)
    saved = pq._fast
    try:
        pq._native()
        if not native:
            pq._fast = False
        want = [[[t.clone() for t in flat(c())] for c in own] for own in calls]
        torch.cuda.synchronize()

        def work(i):
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for r in range(ROUNDS):
                    got = [flat(c()) for c in calls[i]]
                    for k, (a, b) in enumerate(zip(got, want[i])):
                        assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b)), (i, r, k)
                    yield
            s.synchronize()
        failed, done = _run_in_threads(2, work)
    finally:
        pq._fast = saved
    assert not failed, failed[0]
    assert done == [ROUNDS, ROUNDS]
