"""Tensors of over 2^31 elements through the calls whose large offsets no other test reaches: the backward of linear
attention in both types, its fp32 forward, the step's state, and layer norm."""

import pytest

from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_linattn_backward(ss, dtype):
    """v, do and dv of 2.2e9 elements.  A decay of e^-2 a token leaves e^-256 of anything 128 tokens back or ahead: the last
    tokens' outputs equal those of a call on the tail alone, up to where the chunks' borders lie: two roundings each of
    terms up to the largest (2^-6 in bf16, 2^-18 in fp32)."""
    import torch
    L, H, V, K, tail = 270_080, 64, 128, 8, 320
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    gen = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen).to(dt)
    q, k = rnd(1, L, 1, K), rnd(1, L, 1, K)
    v, do = (torch.ones(1, L, H, V, device="cuda", dtype=dt) for _ in range(2))
    v[:, -tail:], do[:, -tail:] = rnd(1, tail, H, V), rnd(1, tail, H, V)
    g = torch.full((H,), -2.0, device="cuda")

    def run(q, k, v, do):
        o, ckpt, h = ss.linattn_fwd(q, k, v, g)
        return {"o": o, "h_last": h} | ss.linattn_bwd(q, k, v, g, ckpt, do)

    big = run(q, k, v, do)
    big = {n: t[:, -100:].clone() if n in ("o", "dq", "dk", "dv") else t for n, t in big.items()}
    small = run(*(t[:, -tail:].contiguous() for t in (q, k, v, do)))
    for n in ("o", "dq", "dk", "dv"):
        want = small[n][:, -100:].float()
        assert (big[n].float() - want).abs().max() <= (2.0 ** -6 if dtype == "bf16" else 2.0 ** -18) * want.abs().max(), n
    assert (big["h_last"] - small["h_last"]).abs().max() <= 2.0 ** -18 * small["h_last"].abs().max()
    assert torch.isfinite(big["dg"]).all()


def test_step(ss):
    """A state of 2.1e9 values: the last sequences equal a call on them alone."""
    import torch
    B, H, K, V, n = 2056, 64, 128, 128, 3
    gen = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=gen)
    q, k, v, g = rnd(B, 8, K), rnd(B, 8, K), rnd(B, H, V), -rnd(B, H).abs()
    h = torch.zeros(B, H, K, V, device="cuda")
    assert h.numel() > 2 ** 31
    h[-n:] = rnd(n, H, K, V)
    s = h[-n:].clone()
    o = ss.linattn_step(q, k, v, g, h)
    so = ss.linattn_step(*(t[-n:].contiguous() for t in (q, k, v, g)), s)
    assert torch.equal(o[-n:], so) and torch.equal(h[-n:], s)
    torch.testing.assert_close(h[0], k[0].repeat_interleave(8, 0)[..., None] * v[0][:, None], rtol=2.0 ** -22, atol=0.0)


@pytest.mark.parametrize("dim", [128, 1024, 8192])
def test_layernorm(ss, dim):
    """x of over 2^31 values in bf16, a width of each kind of kernel: the last rows equal a call on them alone."""
    import torch
    rows = 2 ** 31 // dim + 40
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(64, dim, device="cuda", generator=gen).bfloat16().repeat(rows // 64 + 1, 1)[:rows].contiguous()
    scale, bias = torch.randn(dim, device="cuda", generator=gen), torch.randn(dim, device="cuda", generator=gen)
    assert x.numel() > 2 ** 31
    y, mean, rstd = ss.layernorm_fwd(x, scale, bias, 1e-5)
    cut = lambda t: t[-30:].contiguous()
    y2, mean2, rstd2 = ss.layernorm_fwd(cut(x), scale, bias, 1e-5)
    for a, b in ((y, y2), (mean, mean2), (rstd, rstd2)):
        assert torch.equal(a[-30:], b)
    turns, rest = divmod(rows, 64)
    assert torch.equal(y[(turns - 1) * 64:turns * 64], y[:64])  # rows repeat every 64
    dx, ds, db = ss.layernorm_bwd(x, x, scale, mean, rstd)
    dx2, _, _ = ss.layernorm_bwd(cut(x), cut(x), scale, mean2, rstd2)
    assert torch.equal(dx[-30:], dx2)
    # the column sums: at most 2000 values are added one after another, by a thread and then over threads and CTAs
    f = x[:64].double()
    want = f.sum(0) * turns + f[:rest].sum(0)
    size = f.abs().sum(0) * turns + f[:rest].abs().sum(0)
    assert ((db.double() - want).abs() <= 2.0 ** -24 * 2000 * size).all()
