"""Group norm's statistics where rows are unlike one another: a first position of zeros before data with a mean, a position far from
all others, values that are all alike.

Tolerances as in test_gpu_groupnorm.py, and no wider for any of these: statistics to STEP (2 sqrt(M + 32) + 24), the mean of the
values' root mean square and rstd of itself (an error d of the mean, in deviations, adds d^2 / 2 to it); y is off by the same, and by
the mean's error in deviations."""

import numpy as np
import pytest

from tests.gpu_util import ss_module
from tests.test_gpu_groupnorm import STEP, _near, _np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


SHAPES = [(3, 1, 512, 4), (4, 1, 1024, 2), (3, 8, 64, 4), (200, 6, 128, 8),  # in lanes, and a sample in a CTA
          (2, 600, 64, 4), (4, 2048, 256, 8), (64, 16384, 64, 8), (320, 4096, 8, 1), (1, 30000, 24, 3), (310, 700, 520, 13)]  # in parts


@pytest.mark.parametrize("kind", ["zeros first", "zeros last", "spike first", "spike inside", "one channel", "alike"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,C,groups", SHAPES)
def test_statistics_of_rows_unlike_one_another(ss, N, M, C, groups, dtype, kind):
    import torch
    gen = torch.Generator(device="cuda").manual_seed(M + C)
    x = torch.randn(N, M, C, device="cuda", generator=gen) + 100.0
    if kind == "zeros first":
        x[:, 0] = 0.0
    elif kind == "zeros last":
        x[:, -1] = 0.0
    elif kind == "spike first":
        x = x - 100.0
        x[:, 0] = 700.0
    elif kind == "spike inside":
        x = x - 100.0
        x[:, M // 2, ::2] = -300.0
    elif kind == "one channel":
        x[..., 1] = 5000.0
    else:
        x = torch.full_like(x, 0.1) + (torch.arange(C, device="cuda") % 2) * 0.25
    x = x.to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    scale = torch.ones(C, device="cuda")
    y, mean, rstd = ss.groupnorm_fwd(x, scale, None, groups, 1e-3)
    means, rstds, off = [], [], 0.0
    tol = STEP * (2 * (M + 32) ** 0.5 + 24)
    total = size = 0.0
    for n in range(N):  # float64, a sample at a time
        f = x[n].double().view(M, groups, C // groups)
        m = f.mean((0, 2))
        d = f - m[:, None]
        r = ((d * d).mean((0, 2)) + 1e-3).rsqrt()
        e = d * r[:, None]
        total += float(((y[n].double().view_as(e) - e) ** 2).sum())
        size += float((e * e).sum())
        off = max(off, float((f.square().mean((0, 2)).sqrt() * r).max()))
        means.append(m)
        rstds.append(r)
    _near(mean, _np(torch.stack(means)), tol, "mean", size=float(x.double().square().mean().sqrt()))
    _near(rstd, _np(torch.stack(rstds)), tol + (off * tol) ** 2, "rstd")
    typed = 2.0 ** -8 if dtype == "bf16" else 0.0
    assert total ** 0.5 <= (tol * (1 + off) + typed) * max(size, N * M * C * 1e-6) ** 0.5, (total ** 0.5, size ** 0.5)


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,C", [(1, 8), (1834, 8), (300, 520), (3, 8192), (5, 16384)])
def test_groups_of_one_value(ss, N, C, dtype, silu):
    """A group of one value: y is act(bias) whatever x is, so dx and dscale are 0 and nothing near it, and rstd is eps^(-1/2)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(C + N)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, dy = (3 * torch.randn(N, 1, C, device="cuda", generator=gen).to(dt) for _ in range(2))
    scale, bias = (torch.randn(C, device="cuda", generator=gen) for _ in range(2))
    y, mean, rstd = ss.groupnorm_fwd(x, scale, bias, C, 1e-5, silu=silu)
    b = bias.double()
    want = (b / (1 + torch.exp(-b)) if silu else b).expand(N, 1, C)
    assert torch.equal(mean, x.float()[:, 0])
    assert ((rstd.double() - 1e-5 ** -0.5).abs() <= 4 * 2.0 ** -24 * 1e-5 ** -0.5).all()
    assert ((y.double() - want).abs() <= (2.0 ** -20 + (2.0 ** -8 if dtype == "bf16" else 0.0)) * want.abs()).all()
    dx, dscale, _ = ss.groupnorm_bwd(dy, x, scale, bias, mean, rstd, C, silu=silu)
    assert (dx == 0).all() and (dscale == 0).all()


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,M,C,groups", [(3, 1, 259080, 1016), (2, 1, 65536, 256), (5, 1, 1 << 20, 1 << 17), (2, 3, 40000, 5000), (1, 40, 100000, 2500),
                                          (2, 2, 32776, 8194)])
def test_wide_samples_in_narrow_groups(ss, N, M, C, groups, dtype, silu):
    """More than 32768 channels in groups of at most 256, forward and backward."""
    from oracle.groupnorm import groupnorm_bwd_ref, groupnorm_fwd_ref
    from tests.test_gpu_groupnorm import _case
    d = _case(N, M, C, dtype, seed=C, bias=silu)
    x = _np(d["x"])
    y, mean, rstd = ss.groupnorm_fwd(d["x"], d["scale"], d["bias"], groups, 1e-2, silu=silu)
    ry, rm, rr = groupnorm_fwd_ref(x, _np(d["scale"]), _np(d["bias"]), groups, 1e-2, silu)
    tol, typed = STEP * (2 * (M + 32) ** 0.5 + 24), 2.0 ** -8 if dtype == "bf16" else 0.0
    _near(y, ry, tol + typed, "y")
    _near(mean, rm, tol, "mean", size=np.sqrt(np.mean(x * x)))
    _near(rstd, rr, tol, "rstd")
    dx, ds, db = ss.groupnorm_bwd(d["dy"], d["x"], d["scale"], d["bias"], mean, rstd, groups, silu=silu)
    rdx, rds, rdb = groupnorm_bwd_ref(_np(d["dy"]), x, _np(d["scale"]), _np(d["bias"]), _np(mean), _np(rstd), silu)
    cols = STEP * (4 * (N * M) ** 0.5 + 64)
    _near(dx, rdx, 2 * tol, "dx", size=max(np.sqrt(np.mean(rdx ** 2)), np.sqrt(np.mean(_np(d["dy"]) ** 2)) * np.abs(_np(rstd)).max() if M * (C // groups) < 8 else 0.0))
    _near(ds, rds, cols, "dscale")
    _near(db, rdb, cols, "dbias")
