"""What the gated delta rule's outputs keep beyond a norm over whole outputs: the same bits with and without a checkpoint, roundings
to bf16 that are those of the fp32 result, decay gradients of heads that forget."""

import numpy as np
import pytest

from tests.gpu_util import ss_module
from tests.test_gpu_deltarule import CASES, _case, _fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_a_checkpoint_changes_no_bit(ss, B, L, H, G, K, V, opt, dtype):
    import torch
    d = _case(B, L, H, G, K, V, dtype, seed=L + K + V, **opt)
    o, _, h = _fwd(ss, d)
    o2, _, h2 = _fwd(ss, d, want_ckpt=False)
    assert torch.equal(o, o2) and torch.equal(h, h2)


def test_operands_of_dq_are_rounded_not_cut(ss):
    """bf16 dq = scale e^c do S0^T + E K with u, S0 and E = scale D do u^T as two rounded bf16 terms each, the same in float64, and the
    float64 gradient itself, all rounded to bf16: the kernel's dq is nearer to the first than half of what lies between the first
    and the last.  (What else it rounds, fp32 sums, is 2^-5 of what the terms leave out; cut terms leave out twice as much,
    in other places.)"""
    import torch
    from oracle.deltarule import deltarule_bwd_ref, deltarule_fwd_ref
    from tests.test_gpu_deltarule import _bwd, _np
    L, H, W = 320, 4, 128
    d = _case(1, L, H, H, W, W, "bf16", carry=False, seed=31)
    got = _np(_bwd(ss, d, _fwd(ss, d)[1])["dq"])
    q, k, v, g, beta, do = (_np(d[x]) for x in ("q", "k", "v", "g", "beta", "do"))
    S = deltarule_fwd_ref(q, k, v, g, beta)[1][0]
    bf16 = lambda a: _np(torch.from_numpy(np.ascontiguousarray(a)).bfloat16())

    def two(a):
        a = a.astype(np.float32).astype(np.float64)
        return bf16(a) + bf16(a - bf16(a))

    own = np.zeros((1, L, H, W))
    for h in range(H):
        for t in range(0, L, 64):
            c, at = np.cumsum(g[0, t:t + 64, h]), (0, slice(t, t + 64), h)
            r = np.stack([v[0, i, h] - np.exp(g[0, i, h]) * S[i, h].T @ k[0, i, h] for i in range(t, t + 64)])
            E = W ** -0.5 * np.tril(np.exp(c[:, None] - c)) * (do[at] @ two(beta[at][:, None] * r).T)
            own[at] = W ** -0.5 * np.exp(c)[:, None] * (do[at] @ two(S[t, h]).T) + two(E) @ k[at]
    exact = bf16(deltarule_bwd_ref(q, k, v, g, beta, do)["dq"])
    assert np.linalg.norm(got - bf16(own)) <= 0.5 * np.linalg.norm(bf16(own) - exact)
