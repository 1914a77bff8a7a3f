"""Linear attention on the GPU: each output's root-mean-square distance from the float64 recurrence (bounds and their
derivation in linattn_precision.py; what they tell apart in test_linattn_precision_bounds.py)."""

import numpy as np
import pytest

from oracle.linattn import linattn_bwd_ref, linattn_fwd_ref
from tests.gpu_util import ss_module
from tests.linattn_precision import CASES, bound, inputs, off

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [128, 200])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128), (72, 120), (128, 64)])
@pytest.mark.parametrize("case", CASES)
def test_distance(ss, case, K, V, L, dtype):
    import torch
    d = inputs(case, 2, L, 4, 2, K, V, seed=K + V + L)
    o, S = linattn_fwd_ref(*(d[n] for n in ("q", "k", "v", "g", "h0")))
    ref = {"o": o, "h_last": S[:, -1]} | linattn_bwd_ref(*(d[n] for n in ("q", "k", "v", "g", "do", "h0", "dh_last")))
    act = torch.bfloat16 if dtype == "bf16" else torch.float32
    t = {n: torch.from_numpy(a).to(act if n in ("q", "k", "v", "do") else torch.float32).cuda() for n, a in d.items()}
    o, ckpt, h_last = ss.linattn_fwd(t["q"], t["k"], t["v"], t["g"], h0=t["h0"])
    got = {"o": o, "h_last": h_last} | ss.linattn_bwd(t["q"], t["k"], t["v"], t["g"], ckpt, t["do"], dh_last=t["dh_last"])
    far = {n: (off(got[n].double().cpu().numpy(), r), bound(n, r, dtype)) for n, r in ref.items()}
    print(" ".join(f"{n} {a:.2e}/{b:.2e}" for n, (a, b) in far.items()))
    assert all(a <= b for a, b in far.values()), far


def test_step(ss):
    """The step works in fp32 in both types: h within two roundings of its values, o as an output rounded once."""
    import torch
    d = inputs("state in", 3, 1, 4, 2, 128, 128, seed=7)
    for act, dtype in ((torch.bfloat16, "bf16"), (torch.float32, "f32")):
        t = {n: torch.from_numpy(a).to(act if n in ("q", "k", "v") else torch.float32).cuda() for n, a in d.items()}
        o = ss.linattn_step(*(t[n][:, 0].contiguous() for n in ("q", "k", "v", "g")), t["h0"])
        ro, S = linattn_fwd_ref(*(d[n] for n in ("q", "k", "v", "g", "h0")))
        assert off(t["h0"].double().cpu().numpy(), S[:, -1]) <= 4 * 2.0 ** -24
        a, b = off(o.double().cpu().numpy(), ro[:, 0]), bound("o", ro[:, 0], dtype)
        assert a <= (b if dtype == "f32" else b / 2 ** 0.5), (a, b)
        assert np.isfinite(a)
