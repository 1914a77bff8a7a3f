"""Linear attention whose rows are cut in segments that lie wholly past a row's end: their sums, the join through them
and the walks that only clear outputs and pass a state on.  Tolerances as in test_gpu_linattn.py."""

import pytest

from tests.gpu_util import ss_module
from tests.test_gpu_linattn import _backward, _case, _close, _forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


# B, L, H, G, K, V, options.  Segments are of four chunks at least: 512 tokens in bf16, 256 in fp32
CASES = [
    (3, 1500, 4, 2, 64, 64, {"lengths": [1500, 0, 1]}),
    (4, 1100, 2, 1, 128, 128, {"lengths": [1100, 300, 512, 513]}),
    (3, 1500, 2, 1, 40, 72, {"lengths": [0, 1024, 700], "per_head": True, "packed": True}),
    (2, 1300, 3, 3, 128, 64, {"lengths": [1, 511], "strong": True}),
    (1, 1100, 2, 2, 64, 128, {"lengths": [0], "carry": False}),
]


def _run(ss, d):
    o, ckpt, h = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], lengths=d["lengths"])
    g = ss.linattn_bwd(d["q"], d["k"], d["v"], d["g"], ckpt, d["do"], dh_last=d["dh_last"], lengths=d["lengths"])
    return {"o": o, "h_last": h} | g, ckpt.shape[2]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_segments_past_a_rows_end(ss, B, L, H, G, K, V, opt, dtype):
    import torch
    d = _case(B, L, H, G, K, V, dtype, seed=L + B, **opt)
    got, chunks = _run(ss, d)
    o, S, bo, bS = _forward(d)
    ref, bounds = _backward(d)
    ref |= {"o": o, "h_last": S}
    bounds |= {"o": bo, "h_last": bS}
    for n in ("h_last", "o", "dh0", "dg", "dv", "dq", "dk"):
        _close(got[n], ref[n], bounds[n], (K, V, chunks), dtype, n in ("o", "dq", "dk", "dv"), n)
    again, _ = _run(ss, d)
    assert all(torch.equal(got[n], again[n]) for n in got)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_what_stands_there_is_not_read(ss, dtype):
    import torch
    d = _case(4, 1500, 2, 1, 64, 64, dtype, lengths=[1500, 0, 1, 600], seed=9)
    dead = torch.arange(1500, device="cuda")[None, :] >= d["lengths"][:, None]
    e = dict(d)
    for n, x in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", float("-inf")), ("g", float("nan"))):
        e[n] = torch.where(dead.view(4, 1500, *[1] * (d[n].dim() - 2)), torch.full_like(d[n], x), d[n])
    (a, _), (b, _) = _run(ss, d), _run(ss, e)
    for n in a:
        assert torch.equal(a[n], b[n]), n
    assert torch.equal(b["h_last"][1], d["h0"][1]) and torch.equal(b["dh0"][1], d["dh_last"][1])
    for n in ("o", "dq", "dk", "dv", "dg"):
        assert (b[n][dead] == 0).all(), n
