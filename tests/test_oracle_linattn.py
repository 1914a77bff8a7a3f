"""Pins of the float64 linear attention and layer norm references: against the quadratic form, and their gradients
against central differences."""

import numpy as np
import pytest

from oracle.layernorm import layernorm_bwd_ref, layernorm_fwd_ref
from oracle.linattn import linattn_bwd_ref, linattn_fwd_ref, linattn_step_ref


def _inputs(B, L, H, G, K, V, per_head=False, seed=0):
    r = np.random.default_rng(seed)
    g = -r.uniform(0.01, 1.0, (H,) if per_head else (B, L, H))
    return (r.standard_normal((B, L, G, K)), r.standard_normal((B, L, G, K)), r.standard_normal((B, L, H, V)), g,
            r.standard_normal((B, H, K, V)))


def test_forward_matches_the_quadratic_form():
    q, k, v, g, h0 = _inputs(2, 9, 4, 2, 3, 5)
    o, S = linattn_fwd_ref(q, k, v, g, h0)
    c = np.cumsum(g, 1)
    for b in range(2):
        for h in range(4):
            D = np.tril(np.exp(c[b, :, None, h] - c[b, None, :, h]))
            ref = (q[b, :, h // 2] @ k[b, :, h // 2].T * D) @ v[b, :, h] + np.exp(c[b, :, h])[:, None] * (q[b, :, h // 2] @ h0[b, h])
            np.testing.assert_allclose(o[b, :, h], ref * 3 ** -0.5, rtol=1e-12, atol=1e-12)


def test_steps_and_lengths():
    q, k, v, g, h0 = _inputs(3, 6, 2, 1, 4, 4)
    o, S = linattn_fwd_ref(q, k, v, g, h0, lengths=[6, 0, 1])
    h = h0
    for t in range(6):
        h, ot = linattn_step_ref(h, q[:, t], k[:, t], v[:, t], g[:, t])
        np.testing.assert_allclose(o[0, t], ot[0], rtol=1e-13)
    np.testing.assert_allclose(S[0, -1], h[0], rtol=1e-13)
    assert np.all(S[1, -1] == h0[1]) and np.all(o[1] == 0) and np.all(o[2, 1:] == 0)


@pytest.mark.parametrize("per_head,lengths", [(False, None), (True, None), (False, [5, 0, 2])])
def test_gradient_against_differences(per_head, lengths):
    B, L, H, G, K, V = 3, 5, 4, 2, 3, 2
    q, k, v, g, h0 = _inputs(B, L, H, G, K, V, per_head, seed=1)
    r = np.random.default_rng(2)
    do, dh = r.standard_normal((B, L, H, V)), r.standard_normal((B, H, K, V))

    def loss(q, k, v, g, h0):
        o, S = linattn_fwd_ref(q, k, v, g, h0, lengths=lengths)
        live = np.arange(L)[None, :] < (np.full(B, L) if lengths is None else np.array(lengths))[:, None]
        return np.sum(o * do * live[..., None, None]) + np.sum(S[:, -1] * dh)

    got = linattn_bwd_ref(q, k, v, g, do, h0, dh, lengths=lengths)
    args = {"dq": q, "dk": k, "dv": v, "dg": g, "dh0": h0}
    for i, (name, a) in enumerate(args.items()):
        num = np.zeros_like(a)
        for at in np.ndindex(*a.shape):
            f = []
            for s in (1e-6, -1e-6):
                x = a.copy()
                x[at] += s
                f.append(loss(*[x if j == i else y for j, y in enumerate(args.values())]))
            num[at] = (f[0] - f[1]) / 2e-6
        np.testing.assert_allclose(got[name], num, rtol=1e-6, atol=1e-7, err_msg=name)


def test_layernorm_gradient_against_differences():
    r = np.random.default_rng(3)
    x, dy, scale, bias = r.standard_normal((4, 8)) + 2, r.standard_normal((4, 8)), r.standard_normal(8), r.standard_normal(8)
    _, mean, rstd = layernorm_fwd_ref(x, scale, bias, 1e-5)
    got = layernorm_bwd_ref(dy, x, scale, mean, rstd)
    args = [x, scale, bias]
    for i, a in enumerate(args):
        num = np.zeros_like(a)
        for at in np.ndindex(*a.shape):
            f = []
            for s in (1e-6, -1e-6):
                y = a.copy()
                y[at] += s
                f.append(np.sum(dy * layernorm_fwd_ref(*[y if j == i else z for j, z in enumerate(args)], 1e-5)[0]))
            num[at] = (f[0] - f[1]) / 2e-6
        np.testing.assert_allclose(got[i], num, rtol=1e-6, atol=1e-8)
