"""Group norm with an activation on the GPU against float64.

Tolerance, in the 2-norm of a whole output relative to its own, steps of 2^-24: a statistic is a sum whose terms one thread
adds in sequence at most M of and 32 more follow in trees, whose roundings add like independent ones, sqrt(M + 32), counted twice
(mean and variance); 24 more for the elementwise steps and the hardware's exp2, reciprocals and reciprocal root (2 units each).
Means are held to that of the values' own root mean square; column sums of R rows to 4 sqrt(R) + 64 steps of theirs.  bf16
outputs have their own rounding, at most 2^-8 (eight significant bits: half a step of 2^-7 at a power of two).
"""

import numpy as np
import pytest

from oracle.groupnorm import groupnorm_bwd_ref, groupnorm_fwd_ref
from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.fixture(scope="module")
def ss():
    return ss_module()


def _case(N, M, C, dtype, seed, shift=0.3, bias=True):
    import torch
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cast = lambda a, t=dt: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    f = torch.float32
    return {"x": cast(1.5 * r.standard_normal((N, M, C)) + shift * r.standard_normal((N, 1, C)) + shift), "dy": cast(r.standard_normal((N, M, C))),
            "scale": cast(1 + 0.3 * r.standard_normal(C), f), "bias": cast(0.3 * r.standard_normal(C), f) if bias else None}


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _near(got, ref, tol, name, size=None):
    got = _np(got)
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    off, size = np.linalg.norm(got - ref), np.linalg.norm(ref) if size is None else size * ref.size ** 0.5
    assert off <= tol * size + 1e-30, f"{name}: {off / max(size, 1e-300):.3e} off, {tol:.3e} allowed"


# samples, positions, channels, groups
CASES = [
    (1, 1, 8, 1), (1, 1, 8, 8), (3, 1, 16, 4), (5, 1, 4096, 32), (700, 1, 768, 6), (9, 1, 2048, 8), (2, 1, 24, 3), (40, 1, 520, 13),  # tokens
    (1000, 1, 4096, 1), (3, 1, 8192, 16), (6, 1, 512, 128), (4, 1, 1024, 1),  # tokens, groups past the lanes or below a vector
    (3, 7, 128, 32), (100, 20, 24, 3), (64, 2, 768, 6), (7, 3, 40, 10), (300, 16, 64, 8),  # samples that a CTA holds
    (3, 2, 8192, 8192), (2, 1, 8192, 4096), (5, 4, 2056, 257), (1300, 2, 1024, 16), (3, 5, 72, 9), (4, 60, 200, 25),
    (2, 500, 64, 4), (1, 5000, 512, 1), (9, 33, 4096, 32), (2, 300, 1536, 24), (1, 4, 32768, 8), (1, 1, 32768, 2), (3, 1000, 8, 2),  # in parts
    (2, 129, 4104, 27), (1, 20000, 8, 1), (4, 100, 96, 32),
]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,C,groups", CASES)
def test_forward_and_backward(ss, N, M, C, groups, dtype, silu):
    import torch
    d = _case(N, M, C, dtype, seed=N + M + C, bias=(N + C // 8) % 3 != 0)
    y, mean, rstd = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], groups, 1e-5, silu=silu)
    x = _np(d["x"])
    ry, rm, rr = groupnorm_fwd_ref(x, _np(d["scale"]), _np(d["bias"]), groups, 1e-5, silu)
    tol, typed = STEP * (2 * (M + 32) ** 0.5 + 24), 2.0 ** -8 if dtype == "bf16" else 0.0
    _near(y, ry, tol + typed, "y")
    _near(mean, rm, tol, "mean", size=np.sqrt(np.mean(x * x)))
    _near(rstd, rr, tol, "rstd")
    dx, ds, db = ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], mean, rstd, groups, silu=silu)
    rdx, rds, rdb = groupnorm_bwd_ref(_np(d["dy"]), x, _np(d["scale"]), _np(d["bias"]), _np(mean), _np(rstd), silu)
    cols = STEP * (4 * (N * M) ** 0.5 + 64)
    # (a group of one value or two leaves the difference of what cancels: off by the bound of its terms, w rstd)
    size = max(np.sqrt(np.mean(rdx ** 2)), np.sqrt(np.mean(_np(d["dy"]) ** 2)) * np.abs(_np(rstd)).max() if M * (C // groups) < 8 else 0.0)
    _near(dx, rdx, 2 * tol, "dx", size=size)
    _near(ds, rds, cols, "dscale", size=max(np.sqrt(np.mean(rds ** 2)), 0.1 * (N * M) ** 0.5 if M * (C // groups) < 8 else 0.0))
    _near(db, rdb, cols, "dbias")
    y2, none, none2 = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], groups, 1e-5, silu=silu, want_stats=False)
    assert none is None and none2 is None and torch.equal(y, y2)
    again = ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], mean, rstd, groups, silu=silu)
    assert all(torch.equal(a, b) for a, b in zip(again, (dx, ds, db)))
    # sums accumulate into given tensors, each by itself
    s0, b0 = torch.ones(C, device="cuda"), torch.full((C,), 2.0, device="cuda")
    _, s1, b1 = ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], mean, rstd, groups, silu=silu, dscale=s0.clone())
    assert torch.equal(s1, ds + s0) and torch.equal(b1, db)
    _, s1, b1 = ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], mean, rstd, groups, silu=silu, dbias=b0.clone())
    assert torch.equal(s1, ds) and torch.equal(b1, db + b0)


@pytest.mark.parametrize("M,C,groups", [(1, 256, 4), (1, 512, 1), (8, 64, 4), (600, 64, 4)])
def test_values_far_from_zero(ss, M, C, groups):
    """A mean of 1000 deviations, fp32: mean and variance come of deviations.  x has steps of 2^-14 there, 6e-5 of a deviation."""
    d = _case(4, M, C, "f32", seed=M, shift=0.0)
    d["x"] = d["x"] / 1.5 + 1000.0
    y, mean, rstd = ss.groupnorm_fwd(d["x"], d["scale"], None, groups, 0.0)
    ry, rm, rr = groupnorm_fwd_ref(_np(d["x"]), _np(d["scale"]), None, groups, 0.0)
    tol = STEP * (2 * (M + 32) ** 0.5 + 24)
    _near(mean, rm, tol, "mean")
    # the mean, held to 2^-24 of 1000 and found to the bound of its sum, is off by so much of a deviation
    _near(rstd, rr, 1000 * tol, "rstd")
    _near(y, ry, 2000 * tol, "y")


def test_constant_groups_and_zero_scale(ss):
    """A group of equal values has deviation 0: y is act(bias) and rstd 1 / sqrt(eps); a scale of 0 hides x."""
    import torch
    for M, C, groups in ((1, 64, 4), (5, 64, 4), (900, 64, 4)):
        x = torch.full((2, M, C), 3.0, device="cuda")
        b = torch.linspace(-2, 2, C, device="cuda")
        y, mean, rstd = ss.groupnorm_fwd(x, torch.ones(C, device="cuda"), b, groups, 1e-4, silu=True)
        ref = b.double() / (1 + torch.exp(-b.double()))
        assert (mean == 3.0).all() and ((rstd - 100.0).abs() <= 100 * 4 * 2 ** -23).all()
        assert ((y.double() - ref).abs() <= 2.0 ** -20).all()
        x = torch.randn(2, M, C, device="cuda")
        y, mean, rstd = ss.groupnorm_fwd(x, torch.zeros(C, device="cuda"), None, groups, 1e-4)
        assert (y == 0).all()
        dx, _, db = ss.groupnorm_bwd(torch.ones_like(x), x, torch.zeros(C, device="cuda"), None, mean, rstd, groups)
        assert (dx == 0).all() and (db == 2 * M).all()


def test_large_arguments_of_the_activation(ss):
    """SiLU of +-1000: x and -0, with derivatives 1 and 0, no NaN."""
    import torch
    for M in (1, 4, 700):
        x = torch.randn(2, M, 64, device="cuda")
        scale, bias = torch.full((64,), 0.1, device="cuda"), torch.cat([torch.full((32,), 1000.0), torch.full((32,), -1000.0)]).cuda()
        y, mean, rstd = ss.groupnorm_fwd(x, scale, bias, 2, 1e-5, silu=True)
        dx, ds, db = ss.groupnorm_bwd(torch.ones_like(x), x, scale, bias, mean, rstd, 2, silu=True)
        assert (y[..., :32] > 990).all() and (y[..., 32:] == 0).all()
        assert torch.isfinite(dx).all() and (dx[..., 32:] == 0).all() and (db[:32] == 2 * M).all() and (db[32:] == 0).all()


@pytest.mark.parametrize("M,C,groups", [(1, 512, 4), (1, 512, 1), (6, 64, 4), (900, 64, 4)])
def test_a_bad_value_stays_in_its_sample_and_group(ss, M, C, groups):
    import torch
    d = _case(4, M, C, "bf16", seed=3)
    y, mean, rstd = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], groups, 1e-5, silu=True)
    x = d["x"].clone()
    x[2, M // 2, 5] = float("nan")
    y2, mean2, rstd2 = ss.groupnorm_fwd(x, d["scale"], d["bias"], groups, 1e-5, silu=True)
    cg = C // groups
    assert torch.isnan(y2[2, :, :cg]).all() and torch.isnan(mean2[2, 0])
    keep = torch.ones(4, M, C, dtype=torch.bool, device="cuda")
    keep[2, :, :cg] = False
    assert torch.equal(y2[keep], y[keep])


@pytest.mark.parametrize("shape,groups", [((64, 1, 512), 4), ((64, 1, 512), 1), ((64, 6, 64), 4), ((3, 900, 64), 4)])
def test_on_another_stream_and_from_a_graph(ss, shape, groups):
    import torch
    d = _case(*shape, "bf16", seed=5)

    def both():
        y, m, r = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], groups, 1e-5, silu=True)
        return (y, m, r) + ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], m, r, groups, silu=True)

    want = both()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:  # two at once
        with torch.cuda.stream(s):
            got.append(both())
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(want, g))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    d["x"].mul_(-0.5)
    d["dy"].mul_(2.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(both(), out))


def test_shapes_with_more_positions(ss):
    """x [N, height, width, C] is [N, height * width, C], and [N, C] one position a sample."""
    import torch
    d = _case(3, 35, 32, "f32", seed=7)
    a = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], 4, 1e-5)
    b = ss.groupnorm_fwd(d["x"].view(3, 5, 7, 32), d["scale"], d["bias"], 4, 1e-5)
    assert torch.equal(a[0].view(3, 5, 7, 32), b[0]) and torch.equal(a[1], b[1])
    g = ss.groupnorm_bwd(d["dy"].view(3, 5, 7, 32), d["x"].view(3, 5, 7, 32), d["scale"], d["bias"], a[1], a[2], 4)
    assert g[0].shape == (3, 5, 7, 32)
    c = ss.groupnorm_fwd(d["x"].view(105, 32), d["scale"], d["bias"], 4, 1e-5)
    assert c[0].shape == (105, 32) and c[1].shape == (105, 4)


def test_past_32_bits(ss):
    """Over 2^31 elements, as tokens and as one long sample: the last rows as in a call on them alone."""
    import torch
    C, groups = 1024, 8
    rows = (1 << 31) // C + 4096
    x = torch.ones(rows, 1, C, device="cuda", dtype=torch.bfloat16)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x[-64:] = torch.randn(64, 1, C, device="cuda", generator=gen).bfloat16()
    s, b = torch.rand(C, device="cuda", generator=gen), torch.rand(C, device="cuda", generator=gen)
    y, m, r = ss.groupnorm_fwd(x, s, b, groups, 1e-5, silu=True)
    y2, m2, r2 = ss.groupnorm_fwd(x[-64:].clone(), s, b, groups, 1e-5, silu=True)
    assert torch.equal(y[-64:], y2) and torch.equal(m[-64:], m2) and torch.equal(r[-64:], r2)
    del y
    dx, _, _ = ss.groupnorm_bwd(x, x, s, b, m, r, groups)
    dx2, _, _ = ss.groupnorm_bwd(x[-64:].clone(), x[-64:].clone(), s, b, m2, r2, groups)
    assert torch.equal(dx[-64:], dx2)
    del dx
    y, m, r = ss.groupnorm_fwd(x.view(1, rows, C), s, b, groups, 1e-5)
    f = x[-64:].double().view(64, groups, -1)
    ref = (f - m.double().view(1, groups, 1)) * r.double().view(1, groups, 1) * s.double().view(groups, -1) + b.double().view(groups, -1)
    _near(y[0, -64:], _np(ref).reshape(64, C), 2.0 ** -8, "y")


def test_refusals(ss):
    import torch
    x, w = torch.zeros(4, 3, 16, device="cuda"), torch.ones(16, device="cuda")
    with pytest.raises(ss.SSError, match="status -2"):
        ss.groupnorm_fwd(x, w, w, 3, 1e-5)
    with pytest.raises(ss.SSError, match="status -2"):
        ss.groupnorm_fwd(x, w, w, 4, -1.0)
    with pytest.raises(ss.SSError, match="status -4"):
        ss.groupnorm_fwd(torch.zeros(4, 12, device="cuda"), w[:12].contiguous(), None, 4, 1e-5)
    with pytest.raises(ValueError, match="scale has shape"):
        ss.groupnorm_fwd(x, w[:8].contiguous(), None, 4, 1e-5)
    with pytest.raises(ValueError, match="mean has shape"):
        ss.groupnorm_bwd(x, x, w, w, torch.zeros(4, 8, device="cuda"), torch.zeros(4, 8, device="cuda"), 4)
    with pytest.raises(ss.SSError, match="status -1"):
        ss.groupnorm_fwd(x[:0], w, w, 4, 1e-5)
