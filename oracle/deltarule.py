"""Float64 gated delta rule, step by step from its recurrence:

    r_t = v_t - exp(g_t) S_{t-1}^T k_t,    S_t = exp(g_t) S_{t-1} + beta_t k_t r_t^T,    o_t = scale * S_t^T q_t

q, k [B, L, G, K] serve the H/G heads of a group of v [B, L, H, V]; g (or None) and beta are [B, L, H];
tokens t >= lengths[b] neither decay nor write nor read.  The backward is the adjoint of the same steps.
"""

import numpy as np


def _rows(q, k, v, g, beta, scale, lengths):
    B, L, G, K = q.shape
    H, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    live = np.arange(L)[None, :] < (np.full(B, L) if lengths is None else np.asarray(lengths))[:, None]
    g = np.zeros((B, L, H)) if g is None else np.asarray(g, np.float64)
    e = np.where(live[..., None], np.exp(g), 1.0)
    beta = np.where(live[..., None], np.asarray(beta, np.float64), 0.0)
    cut = lambda a: np.where(live[..., None, None], np.asarray(a, np.float64), 0.0)
    rep = lambda a: np.repeat(cut(a), H // G, axis=2)
    return rep(q), rep(k), cut(v), e, beta, live, scale, (B, L, G, H, K, V)


def deltarule_fwd_ref(q, k, v, g, beta, h0=None, scale=None, lengths=None):
    """-> (o [B, L, H, V], S after every token [B, L+1, H, K, V], the first entry being h0)."""
    q, k, v, e, beta, live, scale, (B, L, G, H, K, V) = _rows(q, k, v, g, beta, scale, lengths)
    S = np.zeros((B, L + 1, H, K, V))
    if h0 is not None:
        S[:, 0] = h0
    o = np.zeros((B, L, H, V))
    for t in range(L):
        D = e[:, t, :, None, None] * S[:, t]
        r = v[:, t] - np.einsum("bhk,bhkv->bhv", k[:, t], D)
        S[:, t + 1] = D + (beta[:, t, :, None] * k[:, t])[..., None] * r[:, :, None]
        o[:, t] = scale * np.einsum("bhk,bhkv->bhv", q[:, t], S[:, t + 1])
    return o, S


def deltarule_bwd_ref(q, k, v, g, beta, do, h0=None, dh_last=None, scale=None, lengths=None):
    """Gradient of sum(o * do) + sum(S_last * dh_last) -> dict dq, dk, dv, dg, dbeta, dh0."""
    _, S = deltarule_fwd_ref(q, k, v, g, beta, h0, scale, lengths)
    q, k, v, e, beta, live, scale, (B, L, G, H, K, V) = _rows(q, k, v, g, beta, scale, lengths)
    do = np.where(live[..., None, None], np.asarray(do, np.float64), 0.0)
    U = np.zeros((B, H, K, V)) if dh_last is None else np.array(dh_last, np.float64)
    dq, dk, dv = np.zeros((B, L, H, K)), np.zeros((B, L, H, K)), np.zeros((B, L, H, V))
    dg, db = np.zeros((B, L, H)), np.zeros((B, L, H))
    for t in range(L - 1, -1, -1):
        D = e[:, t, :, None, None] * S[:, t]
        r = v[:, t] - np.einsum("bhk,bhkv->bhv", k[:, t], D)
        U = U + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", S[:, t + 1], do[:, t])
        Uk = np.einsum("bhkv,bhk->bhv", U, k[:, t])
        db[:, t] = np.einsum("bhv,bhv->bh", Uk, r)
        dr = beta[:, t, :, None] * Uk
        dv[:, t] = dr
        dk[:, t] = beta[:, t, :, None] * np.einsum("bhkv,bhv->bhk", U, r) - np.einsum("bhkv,bhv->bhk", D, dr)
        U = U - k[:, t, :, :, None] * dr[:, :, None]
        dg[:, t] = np.einsum("bhkv,bhkv->bh", D, U)
        U = e[:, t, :, None, None] * U
    dead = ~live[..., None, None]
    share = lambda a: np.where(dead, 0.0, a).reshape(B, L, G, H // G, K).sum(3)
    one = lambda a: np.where(live[..., None], a, 0.0)
    return {"dq": share(dq), "dk": share(dk), "dv": np.where(dead, 0.0, dv), "dg": None if g is None else one(dg), "dbeta": one(db), "dh0": U}


def deltarule_step_ref(h, q, k, v, g, beta, scale=None):
    """One token from state h -> (new h, o)."""
    B, G, K = q.shape
    H = v.shape[1]
    scale = K ** -0.5 if scale is None else scale
    rep = lambda a: np.repeat(np.asarray(a, np.float64), H // G, axis=1)
    e = np.ones((B, H)) if g is None else np.exp(np.asarray(g, np.float64))
    h = e[:, :, None, None] * h
    r = np.asarray(v, np.float64) - np.einsum("bhk,bhkv->bhv", rep(k), h)
    h = h + (np.asarray(beta, np.float64)[..., None] * rep(k))[..., None] * r[:, :, None]
    return h, scale * np.einsum("bhk,bhkv->bhv", rep(q), h)
