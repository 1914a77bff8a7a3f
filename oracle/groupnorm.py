"""Float64 group norm with an activation, channels last: x [N, M, C], statistics over the M positions and the
C / groups channels of a group."""

import numpy as np


def _spread(a, M, C):
    """[N, groups] -> [N, M, C]."""
    return np.broadcast_to(np.repeat(np.asarray(a, np.float64), C // a.shape[1], axis=1)[:, None], (a.shape[0], M, C))


def groupnorm_fwd_ref(x, scale, bias, groups, eps, silu=False):
    """-> (y, mean [N, groups], rstd [N, groups])."""
    x = np.asarray(x, np.float64)
    N, M, C = x.shape
    g = x.reshape(N, M, groups, C // groups)
    mean = g.mean((1, 3))
    rstd = 1.0 / np.sqrt(((g - mean[:, None, :, None]) ** 2).mean((1, 3)) + eps)
    y = (x - _spread(mean, M, C)) * _spread(rstd, M, C) * scale + (0.0 if bias is None else bias)
    return (y / (1.0 + np.exp(-y)) if silu else y), mean, rstd


def groupnorm_bwd_ref(dy, x, scale, bias, mean, rstd, silu=False):
    """-> (dx, dscale, dbias)."""
    x, dy = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    N, M, C = x.shape
    G = mean.shape[1]
    r = _spread(rstd, M, C)
    xh = (x - _spread(mean, M, C)) * r
    if silu:
        t = xh * scale + (0.0 if bias is None else bias)
        p = 1.0 / (1.0 + np.exp(-t))
        dy = dy * p * (1.0 + t * (1.0 - p))
    w = dy * scale
    over = lambda a: _spread(a.reshape(N, M, G, C // G).mean((1, 3)), M, C)
    return r * (w - over(w) - xh * over(w * xh)), (dy * xh).sum((0, 1)), dy.sum((0, 1))
