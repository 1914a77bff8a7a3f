"""Layer norm on the GPU against float64.

Tolerance, element by element (u = 2^-24, n = dim): a sum of n values kept in fp32 is off by at most n u of the sum of
their absolute values (each thread's share and the tree are far shorter; n covers them all).  So with ax = |x| and s = n u + 8 u:
mean by s mean(ax); xh = (x - mean) rstd by (s (ax + mean(ax)) + ...) rstd; the rest follows by the product rule.  y in bf16
is rounded once more (2^-8 of the value).
"""

import numpy as np
import pytest

from oracle.layernorm import layernorm_bwd_ref, layernorm_fwd_ref
from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ss():
    return ss_module()


SHAPES = [(1, 8), (3, 16), (5, 24), (1000, 64), (33, 120), (4097, 128), (7, 248), (100, 256), (65, 264), (517, 768), (9, 1024), (300, 2048),
          (5, 2056), (40, 4104), (700, 8192), (3, 8200), (2, 16384), (3, 32768)]


def _data(rows, dim, dtype, seed):
    import torch
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.from_numpy(r.standard_normal((rows, dim)) + 2.0 * r.standard_normal((rows, 1))).to(dt).cuda()
    dy = torch.from_numpy(r.standard_normal((rows, dim))).to(dt).cuda()
    f = lambda a: torch.from_numpy(a).float().cuda()
    return x, dy, f(1 + 0.1 * r.standard_normal(dim)), f(0.1 * r.standard_normal(dim))


def _np(t):
    return t.double().cpu().numpy()


def _under(got, ref, tol, name):
    got = _np(got)
    assert got.shape == ref.shape and np.all(np.isfinite(got)), name
    over = np.abs(got - ref) > tol
    assert not over.any(), f"{name}: {np.abs(got - ref).max():.3e} off, {over.sum()} values over the bound"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_forward(ss, rows, dim, dtype):
    x, _, scale, bias = _data(rows, dim, dtype, rows + dim)
    for b in (bias, None):
        y, mean, rstd = ss.layernorm_fwd(x, scale, b, 1e-5)
        ry, rm, rr = layernorm_fwd_ref(_np(x), _np(scale), None if b is None else _np(b), 1e-5)
        ax, s = np.abs(_np(x)), (dim + 8) * U
        em = s * ax.mean(1)
        # variance: its summands are off by 2 |x - mean| (em + u |x|), the sum by s; rstd by half of that, relative, and 4 u
        dev = np.abs(_np(x) - rm[:, None])
        ev = (2 * dev * (em[:, None] + U * ax)).mean(1) + em ** 2 + s * (dev ** 2).mean(1)
        er = (0.51 * ev * rr ** 2 + 4 * U) * rr
        _under(mean, rm, em, "mean")
        _under(rstd, rr, er, "rstd")
        ex = (em[:, None] + U * (ax + np.abs(rm)[:, None])) * rr[:, None] + dev * er[:, None]
        tol = (ex + 4 * U * dev * rr[:, None]) * np.abs(_np(scale)) * 1.01 + 4 * U * np.abs(ry) + (0 if b is None else U * np.abs(_np(b)))
        _under(y, ry, tol + (2.0 ** -8 * (np.abs(ry) + tol) if dtype == "bf16" else 0), "y")
    y2, none, none2 = ss.layernorm_fwd(x, scale, None, 1e-5, want_stats=False)
    assert none is None and none2 is None and (y2 == y).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_backward(ss, rows, dim, dtype):
    import torch
    x, dy, scale, _ = _data(rows, dim, dtype, rows * 3 + dim)
    xd = x.double()
    mean, rstd = xd.mean(1).float(), (xd.var(1, unbiased=False) + 1e-5).rsqrt().float()
    dx, ds, db = ss.layernorm_bwd(dy, x, scale, mean, rstd)
    args = [_np(t) for t in (dy, x, scale, mean, rstd)]
    rx, rs, rb = layernorm_bwd_ref(*args)
    g, r = np.abs(args[0]), args[4][:, None]
    xh = np.abs((args[1] - args[3][:, None]) * r) + 2 * U * (np.abs(args[1]) + np.abs(args[3])[:, None]) * r
    exh = 3 * U * (np.abs(args[1]) + np.abs(args[3])[:, None]) * r  # the difference and the product
    w = g * np.abs(args[2])
    s = (dim + 16) * U
    m1, m2 = w.mean(1, keepdims=True), (w * xh).mean(1, keepdims=True)
    e2 = s * m2 + (w * exh).mean(1, keepdims=True)
    _under(dx, rx, 1.01 * r * (8 * U * (w + m1 + xh * m2) + s * m1 + xh * e2 + exh * m2), "dx")
    sr = (rows + 16) * U
    _under(ds, rs, 1.01 * (sr * (g * xh).sum(0) + (g * exh).sum(0)), "dscale")
    _under(db, rb, 1.01 * sr * g.sum(0), "dbias")
    again = ss.layernorm_bwd(dy, x, scale, mean, rstd, dscale=ds.clone(), dbias=db.clone())  # accumulates; same bits
    assert torch.equal(again[0], dx) and torch.equal(again[1], ds + ds) and torch.equal(again[2], db + db)


def test_gradient_against_differences(ss):
    """fp32, along random directions; the loss's rounding is 2^-21 of the sum of its absolute terms over 2 s, its third
    derivative along a unit-size direction within a row's own scale of s^2."""
    import torch
    x, dy, scale, bias = _data(20, 96, "f32", 3)
    gen = torch.Generator(device="cuda").manual_seed(2)
    y, mean, rstd = ss.layernorm_fwd(x, scale, bias, 1e-5)
    grads = dict(zip(("x", "scale", "bias"), ss.layernorm_bwd(dy, x, scale, mean, rstd)))
    base = {"x": x, "scale": scale, "bias": bias}
    loss = lambda a: float((ss.layernorm_fwd(a["x"], a["scale"], a["bias"], 1e-5)[0].double() * dy.double()).sum())
    size = float((y.abs() * dy.abs()).sum())
    s = 2.0 ** -7
    for n, t in base.items():
        u = torch.randn(t.shape, device="cuda", generator=gen)
        slope = (loss(base | {n: t + s * u}) - loss(base | {n: t - s * u})) / (2 * s)
        want = float((grads[n].double() * u.double()).sum())
        assert abs(slope - want) <= 2.0 ** -21 * size / s + 4 * s * s * size, n


def test_rows_of_one_value_and_graph(ss):
    """A row whose values are all equal has y = bias; the calls can be captured, also on another stream."""
    import torch
    x = torch.full((6, 320), 3.0, device="cuda")
    scale, bias = torch.full((320,), 2.0, device="cuda"), torch.linspace(-1, 1, 320, device="cuda")
    y, mean, rstd = ss.layernorm_fwd(x, scale, bias, 1e-5)
    assert torch.equal(y, bias.expand(6, 320)) and (mean == 3.0).all()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        y2, m2, r2 = ss.layernorm_fwd(x, scale, bias, 1e-5)
        d2 = ss.layernorm_bwd(y2, x, scale, m2, r2)
    x.copy_(torch.randn(6, 320, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    graph.replay()
    y3, m3, r3 = ss.layernorm_fwd(x, scale, bias, 1e-5)
    d3 = ss.layernorm_bwd(y3, x, scale, m3, r3)
    torch.cuda.synchronize()
    assert torch.equal(y2, y3) and all(torch.equal(a, b) for a, b in zip(d2, d3))


def test_refusals(ss):
    import torch
    x, s = torch.zeros(4, 16, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(ValueError, match="scale has shape"):
        ss.layernorm_fwd(x, s[:8], None, 1e-5)
    with pytest.raises(ValueError, match="contiguous"):
        ss.layernorm_fwd(x.t(), torch.ones(4, device="cuda"), None, 1e-5)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ss.layernorm_fwd(x.half(), s, None, 1e-5)
    with pytest.raises(ss.SSError, match="status -4"):
        ss.layernorm_fwd(x[:, :12].contiguous(), s[:12], None, 1e-5)
    with pytest.raises(ss.SSError, match="status -2"):
        ss.layernorm_fwd(x, s, None, -1.0)
    with pytest.raises(ss.SSError, match="status -1"):  # an empty tensor has no memory
        ss.layernorm_fwd(x[:0], s, None, 1e-5)
    with pytest.raises(ValueError, match="mean has shape"):
        ss.layernorm_bwd(x, x, s, torch.zeros(3, device="cuda"), torch.zeros(4, device="cuda"))
