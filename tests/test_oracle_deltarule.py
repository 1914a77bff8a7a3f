"""Pins of the float64 gated delta rule and group norm references: closed forms, and their gradients against central
differences."""

import numpy as np
import pytest

from oracle.deltarule import deltarule_bwd_ref, deltarule_fwd_ref, deltarule_step_ref
from oracle.groupnorm import groupnorm_bwd_ref, groupnorm_fwd_ref
from oracle.layernorm import layernorm_bwd_ref, layernorm_fwd_ref
from oracle.linattn import linattn_fwd_ref


def _inputs(B, L, H, G, K, V, seed=0):
    r = np.random.default_rng(seed)
    k = r.standard_normal((B, L, G, K))
    return (r.standard_normal((B, L, G, K)), k / np.linalg.norm(k, axis=-1, keepdims=True), r.standard_normal((B, L, H, V)),
            -r.uniform(0.01, 1.0, (B, L, H)), r.uniform(0.1, 1.9, (B, L, H)), r.standard_normal((B, H, K, V)))


def test_orthonormal_keys_store_and_replace():
    """Without decays and with beta = 1, the state answers a key with the value written last under it."""
    K, V = 4, 3
    k = np.eye(K)[[0, 1, 2, 3, 1]].reshape(1, 5, 1, K)
    v = np.random.default_rng(0).standard_normal((1, 5, 1, V))
    _, S = deltarule_fwd_ref(k, k, v, None, np.ones((1, 5, 1)))
    np.testing.assert_allclose(S[0, -1, 0], v[0, [0, 4, 2, 3], 0], rtol=1e-14)


def test_a_transition_matrix_for_each_token():
    """S_t = exp(g)(I - beta k k^T) S_{t-1} + beta k v^T."""
    q, k, v, g, beta, h0 = _inputs(2, 7, 4, 2, 3, 5)
    _, S = deltarule_fwd_ref(q, k, v, g, beta, h0)
    for b in range(2):
        for h in range(4):
            X = h0[b, h]
            for t in range(7):
                kk, bt = k[b, t, h // 2], beta[b, t, h]
                X = np.exp(g[b, t, h]) * (np.eye(3) - bt * np.outer(kk, kk)) @ X + bt * np.outer(kk, v[b, t, h])
            np.testing.assert_allclose(S[b, -1, h], X, rtol=1e-12, atol=1e-12)


def test_small_writes_are_linear_attention():
    """To first order in beta the write is beta k v^T."""
    q, k, v, g, beta, _ = _inputs(1, 6, 2, 1, 4, 4, seed=1)
    s = 1e-6
    o, _ = deltarule_fwd_ref(q, k, v, g, s * beta)
    ref, _ = linattn_fwd_ref(q, k, v * (s * beta)[..., None], g)
    np.testing.assert_allclose(o, ref, rtol=0, atol=50 * s * s)


def test_steps_and_lengths():
    q, k, v, g, beta, h0 = _inputs(3, 6, 2, 1, 4, 4)
    o, S = deltarule_fwd_ref(q, k, v, g, beta, h0, lengths=[6, 0, 1])
    h = h0
    for t in range(6):
        h, ot = deltarule_step_ref(h, q[:, t], k[:, t], v[:, t], g[:, t], beta[:, t])
        np.testing.assert_allclose(o[0, t], ot[0], rtol=1e-13)
    np.testing.assert_allclose(S[0, -1], h[0], rtol=1e-13)
    assert np.all(S[1, -1] == h0[1]) and np.all(o[1] == 0) and np.all(o[2, 1:] == 0)


def _differences(loss, args, i, s=1e-6):
    num = np.zeros_like(args[i])
    for at in np.ndindex(*args[i].shape):
        f = []
        for d in (s, -s):
            x = args[i].copy()
            x[at] += d
            f.append(loss(*[x if j == i else y for j, y in enumerate(args)]))
        num[at] = (f[0] - f[1]) / (2 * s)
    return num


@pytest.mark.parametrize("lengths", [None, [5, 0, 2]])
def test_gradient_against_differences(lengths):
    B, L, H, G, K, V = 3, 5, 4, 2, 3, 2
    args = list(_inputs(B, L, H, G, K, V, seed=1))
    r = np.random.default_rng(2)
    do, dh = r.standard_normal((B, L, H, V)), r.standard_normal((B, H, K, V))
    live = np.arange(L)[None, :] < (np.full(B, L) if lengths is None else np.array(lengths))[:, None]

    def loss(q, k, v, g, beta, h0):
        o, S = deltarule_fwd_ref(q, k, v, g, beta, h0, lengths=lengths)
        return np.sum(o * do * live[..., None, None]) + np.sum(S[:, -1] * dh)

    got = deltarule_bwd_ref(*args[:5], do, args[5], dh, lengths=lengths)
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dh0")):
        np.testing.assert_allclose(got[name], _differences(loss, args, i), rtol=1e-6, atol=1e-7, err_msg=name)


@pytest.mark.parametrize("silu", [False, True])
def test_groupnorm_gradient_against_differences(silu):
    r = np.random.default_rng(3)
    x, dy, scale, bias = r.standard_normal((2, 3, 6)) + 2, r.standard_normal((2, 3, 6)), r.standard_normal(6), r.standard_normal(6)
    _, mean, rstd = groupnorm_fwd_ref(x, scale, bias, 3, 1e-5, silu)
    got = groupnorm_bwd_ref(dy, x, scale, bias, mean, rstd, silu)
    loss = lambda x, s, b: np.sum(dy * groupnorm_fwd_ref(x, s, b, 3, 1e-5, silu)[0])
    for i, name in enumerate(("dx", "dscale", "dbias")):
        np.testing.assert_allclose(got[i], _differences(loss, [x, scale, bias], i), rtol=1e-6, atol=1e-7, err_msg=name)


def test_one_group_of_one_position_is_layer_norm():
    r = np.random.default_rng(4)
    x, dy, scale, bias = r.standard_normal((5, 8)), r.standard_normal((5, 8)), r.standard_normal(8), r.standard_normal(8)
    y, mean, rstd = groupnorm_fwd_ref(x[:, None], scale, bias, 1, 1e-5)
    ref = layernorm_fwd_ref(x, scale, bias, 1e-5)
    for a, b in zip((y[:, 0], mean[:, 0], rstd[:, 0]), ref):
        np.testing.assert_allclose(a, b, rtol=1e-13)
    for a, b in zip(groupnorm_bwd_ref(dy[:, None], x[:, None], scale, bias, mean, rstd), layernorm_bwd_ref(dy, x, scale, *ref[1:])):
        np.testing.assert_allclose(np.squeeze(a), b, rtol=1e-12, atol=1e-13)
