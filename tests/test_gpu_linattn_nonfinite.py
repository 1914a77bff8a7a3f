"""A NaN or infinity in a live token of linear attention: what it must reach, and what keeps its bits."""

import pytest

from tests.gpu_util import ss_module
from tests.test_gpu_linattn import _case

pytestmark = pytest.mark.gpu
T = 150  # in the tokens 128 .. 191 of a chunk of 64, 128 .. 255 of one of 128


@pytest.fixture(scope="module")
def ss():
    return ss_module()


def _run(ss, d):
    o, ckpt, h = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"])
    g = ss.linattn_bwd(d["q"], d["k"], d["v"], d["g"], ckpt, d["do"], dh_last=d["dh_last"])
    return {"o": o, "h_last": h} | g


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("V", [64, 128])
@pytest.mark.parametrize("name,value", [("q", float("nan")), ("k", float("inf")), ("k", float("nan")), ("v", float("inf")), ("v", float("nan")),
                                        ("do", float("-inf")), ("g", float("nan"))])
def test_live_token(ss, name, value, V, dtype):
    import torch
    H, G = 4, 2
    d = _case(2, 300, H, G, 64, V, dtype, seed=3)
    e = dict(d)
    e[name] = d[name].clone()
    at = 1 if name in ("v", "do", "g") else 0  # head 1, or group 0 of heads 0 and 1
    e[name][(0, T, at, 5) if name != "g" else (0, T, at)] = value
    heads = [at] if name in ("v", "do", "g") else [0, 1]
    a, b = _run(ss, d), _run(ss, e)
    others = [h for h in range(H) if h not in heads]
    for n in a:
        assert torch.equal(a[n][1], b[n][1]), f"{n}: another batch row"
    for n in ("o", "dv", "dg"):
        assert torch.equal(a[n][0][:, others], b[n][0][:, others]), f"{n}: another head"
    for n in ("h_last", "dh0"):
        assert torch.equal(a[n][0][others], b[n][0][others]), f"{n}: another head"
    for n in ("dq", "dk"):
        assert torch.equal(a[n][0][:, 1], b[n][0][:, 1]), f"{n}: another group"
    assert torch.equal(a["o"][0, :128], b["o"][0, :128]), "o: an earlier chunk"
    bad = lambda t: ~torch.isfinite(t)
    if name == "do":
        assert torch.equal(a["o"], b["o"]) and torch.equal(a["h_last"], b["h_last"])
        assert bad(b["dq"][0, T, 0]).any() and bad(b["dv"][0, :T + 1, at, 5]).all() and bad(b["dh0"][0, at, :, 5]).all()
        return
    if name == "q":
        assert bad(b["o"][0, T, heads]).all() and torch.equal(a["h_last"], b["h_last"])
        keep = [t for t in range(300) if t != T]
        assert torch.equal(a["o"][0, keep], b["o"][0, keep])
        return
    columns = [5] if name == "v" else list(range(V))
    rows = [5] if name == "k" else list(range(64))
    assert bad(b["o"][0, T:, heads][..., columns]).all(), "o from the token on"
    assert bad(b["h_last"][0, heads][:, rows][..., columns]).all(), "h_last"
