"""Float64 layer norm: y = (x - mean) * rstd * scale + bias per row, and its gradient."""

import numpy as np


def layernorm_fwd_ref(x, scale, bias, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * scale
    return (y if bias is None else y + bias), mean, rstd


def layernorm_bwd_ref(dy, x, scale, mean, rstd):
    """-> (dx, dscale, dbias) for the given statistics."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    r = np.asarray(rstd, np.float64)[:, None]
    xh = (x - np.asarray(mean, np.float64)[:, None]) * r
    w = dy * scale
    dx = r * (w - w.mean(1, keepdims=True) - xh * (w * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
