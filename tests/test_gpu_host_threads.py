"""Calls from several host threads at once, each on its own stream: sizes whose launches ask for different amounts of shared memory
must not take it from one another."""

import threading

import pytest

from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


def _together(works, rounds):
    """Each of `works` in a thread with a stream of its own, all starting together; their results of the first and last round."""
    import torch
    start, got, failed = threading.Barrier(len(works)), [None] * len(works), []

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                first = works[i]()
                for _ in range(rounds):
                    last = works[i]()
                torch.cuda.current_stream().synchronize()
                got[i] = (first, last)
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(works))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    return got


def _same(a, b):
    import torch
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_delta_rule_of_two_sizes(ss):
    import torch
    from tests.test_gpu_deltarule import _bwd, _case, _fwd

    def work(K, V):
        d = _case(1, 40, 2, 1, K, V, "f32", seed=K + V)

        def go():
            o, ckpt, h = _fwd(ss, d)
            g = _bwd(ss, d, ckpt)
            return [o, h] + [g[n] for n in ("dq", "dk", "dv", "dg", "dbeta", "dh0")]
        return go

    works = [work(64, 8), work(64, 128), work(40, 72), work(128, 16), work(96, 128)]
    want = [w() for w in works]
    torch.cuda.synchronize()
    for (first, last), w in zip(_together(works, 150), want):
        assert _same(first, w) and _same(last, w)


def _many(calls, rounds=4000):
    """Each of `calls` made over and over in a thread of its own; the statuses that came back."""
    import ctypes
    import torch
    start, seen = threading.Barrier(len(calls)), [set() for _ in calls]
    streams = [torch.cuda.Stream() for _ in calls]

    def run(i):
        fn, args = calls[i]
        args = [*args, ctypes.c_void_p(streams[i].cuda_stream)]
        start.wait()
        for _ in range(rounds):
            seen[i].add(fn(*args))

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return set().union(*seen)


def test_launches_keep_their_shared_memory(ss):
    """A small and a large call of the same kernels, launched without a pause between: every one succeeds."""
    import torch
    lib = ss.load()
    p = lambda t: t.data_ptr()  # noqa: E731
    keep, calls = [], []
    for N, M, C, groups in ((1, 2, 16, 2), (1, 2, 8192, 8192), (1, 3, 64, 4), (1, 2, 4096, 16)):
        x, w, st = torch.randn(N, M, C, device="cuda").bfloat16(), torch.ones(C, device="cuda"), torch.ones(2, N, groups, device="cuda")
        keep += [x, w, st, torch.empty_like(x)]
        calls.append((lib.groupnorm_fwd, (p(x), p(w), None, 1e-5, p(keep[-1]), p(st[0]), p(st[1]), N, M, C, groups, 0, 1, None, 0)))
    assert _many(calls) == {0}
    calls = []
    for rows, dim in ((3, 1024), (3, 8192), (3, 4096), (3, 2048)):
        x, w, y = torch.randn(rows, dim, device="cuda"), torch.ones(dim, device="cuda"), torch.empty(rows, dim, device="cuda")
        keep += [x, w, y, torch.empty(rows, device="cuda")]
        calls.append((lib.rmsnorm_fwd, (p(x), p(w), 1e-5, p(y), p(keep[-1]), rows, dim, 0)))
    assert _many(calls) == {0}
    calls = []
    for K, V in ((64, 8), (64, 128), (64, 16), (64, 104)):
        q, v = torch.randn(1, 8, 1, K, device="cuda"), torch.randn(1, 8, 1, V, device="cuda")
        b, ws = torch.ones(1, 8, 1, device="cuda"), torch.empty(1 << 20, device="cuda", dtype=torch.uint8)
        keep += [q, v, b, ws, torch.empty_like(v)]
        calls.append((lib.deltarule_fwd, (p(q), K, p(q), K, p(v), V, None, p(b), None, None, p(keep[-1]), None, None, 1, 8, 1, 1, K, V, 1.0, 0,
                                          p(ws), 1 << 20)))
    assert _many(calls) == {0}


def test_group_norm_of_two_sizes(ss):
    import torch
    from tests.test_gpu_groupnorm import _case

    def work(N, M, C, groups):
        d = _case(N, M, C, "bf16", seed=M + C)

        def go():
            y, m, r = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], groups, 1e-5, silu=True)
            return [y, m, r, *ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], m, r, groups, silu=True)]
        return go

    works = [work(4, 2, 8192, 8192), work(4, 3, 64, 4), work(4, 8, 2048, 16), work(4, 2, 16, 2)]
    want = [w() for w in works]
    torch.cuda.synchronize()
    for (first, last), w in zip(_together(works, 300), want):
        assert _same(first, w) and _same(last, w)
