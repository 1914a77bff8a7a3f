"""Float64 linear attention with a decay for each head, step by step from its recurrence:

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,    o_t = scale * S_t^T q_t

q, k [B, L, G, K] serve the H/G heads of a group of v [B, L, H, V]; g is [B, L, H] or [H];
tokens t >= lengths[b] neither decay nor add nor read.  The backward is the adjoint of the same steps.
"""

import numpy as np


def _rows(q, k, v, g, scale, lengths):
    B, L, G, K = q.shape
    H, V = v.shape[2:]
    scale = K ** -0.5 if scale is None else scale
    live = np.arange(L)[None, :] < (np.full(B, L) if lengths is None else np.asarray(lengths))[:, None]
    e = np.exp(np.broadcast_to(np.asarray(g, np.float64), (B, L, H)))
    e = np.where(live[..., None], e, 1.0)
    cut = lambda a: np.where(live[..., None, None], np.asarray(a, np.float64), 0.0)
    rep = lambda a: np.repeat(cut(a), H // G, axis=2)
    return rep(q), rep(k), cut(v), e, live, scale, (B, L, G, H, K, V)


def linattn_fwd_ref(q, k, v, g, h0=None, scale=None, lengths=None):
    """-> (o [B, L, H, V], S after every token [B, L+1, H, K, V], the first entry being h0)."""
    q, k, v, e, live, scale, (B, L, G, H, K, V) = _rows(q, k, v, g, scale, lengths)
    S = np.zeros((B, L + 1, H, K, V))
    if h0 is not None:
        S[:, 0] = h0
    o = np.zeros((B, L, H, V))
    for t in range(L):
        S[:, t + 1] = e[:, t, :, None, None] * S[:, t] + k[:, t, :, :, None] * v[:, t, :, None, :]
        o[:, t] = scale * np.einsum("bhk,bhkv->bhv", q[:, t], S[:, t + 1])
    return o, S


def linattn_bwd_ref(q, k, v, g, do, h0=None, dh_last=None, scale=None, lengths=None):
    """Gradient of sum(o * do) + sum(S_last * dh_last) -> dict dq, dk, dv, dg, dh0."""
    per_head = np.ndim(g) == 1
    _, S = linattn_fwd_ref(q, k, v, g, h0, scale, lengths)
    q, k, v, e, live, scale, (B, L, G, H, K, V) = _rows(q, k, v, g, scale, lengths)
    do = np.where(live[..., None, None], np.asarray(do, np.float64), 0.0)
    U = np.zeros((B, H, K, V)) if dh_last is None else np.array(dh_last, np.float64)
    dq, dk, dv, dg = np.zeros((B, L, H, K)), np.zeros((B, L, H, K)), np.zeros((B, L, H, V)), np.zeros((B, L, H))
    for t in range(L - 1, -1, -1):
        U = U + scale * q[:, t, :, :, None] * do[:, t, :, None, :]
        dq[:, t] = scale * np.einsum("bhkv,bhv->bhk", S[:, t + 1], do[:, t])
        dk[:, t] = np.einsum("bhkv,bhv->bhk", U, v[:, t])
        dv[:, t] = np.einsum("bhkv,bhk->bhv", U, k[:, t])
        dg[:, t] = e[:, t] * np.einsum("bhkv,bhkv->bh", S[:, t], U)
        U = e[:, t, :, None, None] * U
    dead = ~live[..., None, None]
    share = lambda a: np.where(dead, 0.0, a).reshape(B, L, G, H // G, K).sum(3)
    dg = np.where(live[..., None], dg, 0.0)
    return {"dq": share(dq), "dk": share(dk), "dv": np.where(dead, 0.0, dv), "dg": dg.sum((0, 1)) if per_head else dg, "dh0": U}


def linattn_step_ref(h, q, k, v, g, scale=None):
    """One token from state h -> (new h, o)."""
    B, G, K = q.shape
    H = v.shape[1]
    scale = K ** -0.5 if scale is None else scale
    rep = lambda a: np.repeat(np.asarray(a, np.float64), H // G, axis=1)
    e = np.exp(np.broadcast_to(np.asarray(g, np.float64), (B, H)))
    h = e[:, :, None, None] * h + rep(k)[..., None] * np.asarray(v, np.float64)[:, :, None, :]
    return h, scale * np.einsum("bhk,bhkv->bhv", rep(q), h)
