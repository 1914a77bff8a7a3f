"""What the gated delta rule's outputs keep beyond a norm over whole outputs: the same bits with and without a checkpoint, roundings
to bf16 that are those of the fp32 result, decay gradients of heads that forget."""

import numpy as np
import pytest

from tests.gpu_util import ss_module
from tests.test_gpu_deltarule import CASES, _case, _fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_a_checkpoint_changes_no_bit(ss, B, L, H, G, K, V, opt, dtype):
    import torch
    d = _case(B, L, H, G, K, V, dtype, seed=L + K + V, **opt)
    o, _, h = _fwd(ss, d)
    o2, _, h2 = _fwd(ss, d, want_ckpt=False)
    assert torch.equal(o, o2) and torch.equal(h, h2)


def test_operands_of_dq_are_rounded_not_cut(ss):
    """bf16 dq = scale e^c do S0^T + E K with u, S0 and E = scale D do u^T as two rounded bf16 terms each, the same in float64, and the
    float64 gradient itself, all rounded to bf16: the kernel's dq is nearer to the first than half of what lies between the first
    and the last.  (What else it rounds, fp32 sums, is 2^-5 of what the terms leave out; cut terms leave out twice as much,
    in other places.)"""
    import torch
    from oracle.deltarule import deltarule_bwd_ref, deltarule_fwd_ref
    from tests.test_gpu_deltarule import _bwd, _np
    L, H, W = 320, 4, 128
    d = _case(1, L, H, H, W, W, "bf16", carry=False, seed=31)
    got = _np(_bwd(ss, d, _fwd(ss, d)[1])["dq"])
    q, k, v, g, beta, do = (_np(d[x]) for x in ("q", "k", "v", "g", "beta", "do"))
    S = deltarule_fwd_ref(q, k, v, g, beta)[1][0]
    bf16 = lambda a: _np(torch.from_numpy(np.ascontiguousarray(a)).bfloat16())

    def two(a):
        a = a.astype(np.float32).astype(np.float64)
        return bf16(a) + bf16(a - bf16(a))

    own = np.zeros((1, L, H, W))
    for h in range(H):
        for t in range(0, L, 64):
            c, at = np.cumsum(g[0, t:t + 64, h]), (0, slice(t, t + 64), h)
            r = np.stack([v[0, i, h] - np.exp(g[0, i, h]) * S[i, h].T @ k[0, i, h] for i in range(t, t + 64)])
            E = W ** -0.5 * np.tril(np.exp(c[:, None] - c)) * (do[at] @ two(beta[at][:, None] * r).T)
            own[at] = W ** -0.5 * np.exp(c)[:, None] * (do[at] @ two(S[t, h]).T) + two(E) @ k[at]
    exact = bf16(deltarule_bwd_ref(q, k, v, g, beta, do)["dq"])
    assert np.linalg.norm(got - bf16(own)) <= 0.5 * np.linalg.norm(bf16(own) - exact)


LEVELS = [-0.01, -0.3, -1.0, -1.9, -2.1, -4.0, -8.0, -12.0, -16.0, -30.0, -200.0]


def _forgetting(L, dtype, mixed, K=48, V=40, seed=0):
    """A head for each level of its log decays, within a tenth; or among weak ones with now and then a token at the level."""
    import torch
    r = np.random.default_rng(seed)
    d = _case(2, L, len(LEVELS), 1, K, V, dtype, seed=seed)
    g = np.array(LEVELS) * r.uniform(0.9, 1.1, (2, L, len(LEVELS)))
    if mixed:
        at = r.random(g.shape) < 0.1
        g = np.where(at, g, -np.exp(r.uniform(np.log(1e-3), np.log(0.3), g.shape)))
    else:
        at = np.ones(g.shape, bool)
    d["g"] = torch.from_numpy(g).float().cuda()
    return d, at


@pytest.mark.parametrize("mixed", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L", [1, 3, 64, 200])
def test_decay_gradients_of_heads_that_forget(ss, L, dtype, mixed):
    """dg of each level by itself.  dg_t carries e^{g_t}; a form in which each token's own write cancels keeps the rounding of terms
    of any size.  fp32: the three-fold bound of a gradient, 3 F, at every level.  bf16: where g is below -2 the sum of what
    crosses the token, with products of two operands that are off by 2^-16 each and drop as much, 3 * 2^-16; above, the other form,
    whose terms are at most e^2 of the result: 3 F e^2."""
    from oracle.deltarule import deltarule_bwd_ref
    from tests.test_gpu_deltarule import _bwd, _near, _np, _tol
    d, at = _forgetting(L, dtype, mixed, seed=L)
    got = _np(_bwd(ss, d, _fwd(ss, d)[1])["dg"])
    ref = deltarule_bwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "beta", "do", "h0", "dh_last")])["dg"]
    tol = _tol(L, dtype, False, 3) * (np.exp(2) if dtype == "bf16" else 1.0) + (3 * 2.0 ** -16 if dtype == "bf16" else 0.0)
    for i, level in enumerate(LEVELS):
        for group in (at[..., i], ~at[..., i]):
            if group.any():
                a, b = got[..., i][group], ref[..., i][group]
                off, size = np.linalg.norm(a - b), np.linalg.norm(b)
                assert off <= tol * size + 1e-30, (level, off / max(size, 1e-300), tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_decay_gradients_that_forget_in_every_layout(ss, dtype):
    """The sizes, strides, shared heads, lengths and dead tokens of the other tests, each head with its own level; NaN past the ends;
    twice the same bits."""
    import torch
    from oracle.deltarule import deltarule_bwd_ref
    from tests.test_gpu_deltarule import _bwd, _np, _tol
    for B, L, H, G, K, V, opt in CASES:
        if opt.get("decay") is False or opt.get("strong"):
            continue
        d = _case(B, L, H, G, K, V, dtype, seed=L, **opt)
        d["g"] = torch.tensor(([-9.0, -0.5, -20.0] * H)[:H], device="cuda") * (0.9 + 0.2 * torch.rand(B, L, H, device="cuda"))
        n = None if d["lengths"] is None else np.clip(_np(d["lengths"]), 0, L)
        dead = None
        if n is not None:
            dead = torch.arange(L, device="cuda")[None, :] >= torch.tensor(n, device="cuda")[:, None]
            for name in ("q", "k", "v", "do", "g", "beta"):
                d[name] = torch.where(dead.view(B, L, *[1] * (d[name].dim() - 2)), torch.full_like(d[name], float("nan")), d[name])
        ckpt = _fwd(ss, d)[1]
        got = _bwd(ss, d, ckpt)["dg"]
        assert torch.equal(got, _bwd(ss, d, ckpt)["dg"])
        assert dead is None or (got[dead] == 0).all()
        ref = deltarule_bwd_ref(*[np.nan_to_num(_np(d[x])) if d[x] is not None else None for x in ("q", "k", "v", "g", "beta", "do", "h0", "dh_last")], lengths=n)["dg"]
        tol = _tol(L, dtype, False, 3) * (np.exp(2) if dtype == "bf16" else 1.0) + (3 * 2.0 ** -16 if dtype == "bf16" else 0.0)
        for h in range(H):
            off, size = np.linalg.norm(_np(got)[..., h] - ref[..., h]), np.linalg.norm(ref[..., h])
            assert off <= tol * size + 1e-30, (B, L, H, K, V, h, off / max(size, 1e-300), tol)
    assert ss.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("power", [-100, -80, -66, -30, 30, 66, 90])
def test_values_and_gradients_of_any_size(ss, dtype, power):
    """The forward is linear in q and in (v, h0), the backward in (do, dh_last): scaled by a power of two, each gives its results scaled
    alike.  Beside 2^-100 the smallest terms of an operand, 2^-24 of it, are near the least normal number, and bf16 ones past
    it: 2^-8 and 2^-16 of them are subnormal."""
    import torch
    from tests.test_gpu_deltarule import _bwd, _near, _np, _tol
    d = _case(2, 150, 4, 2, 48, 40, dtype, seed=4)
    f = 2.0 ** power
    o, ckpt, h = _fwd(ss, d)
    g = _bwd(ss, d, ckpt)
    alone = _bwd(ss, d | {"dh_last": None}, ckpt)
    tol = _tol(150, dtype, False, 3) * 2 + (2.0 ** -7 if dtype == "bf16" else 0.0)  # two results that round apart
    e = d | {"do": d["do"] * f, "dh_last": d["dh_last"] * f}
    for n, t in _bwd(ss, e, ckpt).items():
        _near(t.double() / f, _np(g[n]), tol, f"do: {n}")
    e = d | {"q": d["q"] * f}
    o2, ckpt2, h2 = _fwd(ss, e)
    assert torch.equal(h2, h)
    _near(o2.double() / f, _np(o), tol, "q: o")
    for n, t in _bwd(ss, e | {"dh_last": None}, ckpt2).items():
        _near(t.double() / (1.0 if n == "dq" else f), _np(alone[n]), tol, f"q: {n}")
    e = d | {"v": d["v"] * f, "h0": d["h0"] * f}
    o2, ckpt2, h2 = _fwd(ss, e)
    _near(o2.double() / f, _np(o), tol, "v: o")
    _near(h2.double() / f, _np(h), tol, "v: h")
    for n, t in _bwd(ss, e, ckpt2).items():
        _near(t.double() / (1.0 if n in ("dv", "dh0") else f), _np(g[n]), tol, f"v: {n}")


@pytest.mark.parametrize("seed", [1, 2, 3])
@pytest.mark.parametrize("K,V", [(64, 64), (128, 128)])
def test_fp32_sums_are_cut_once_a_step(ss, K, V, seed):
    """fp32, no decay, beta up to 2.  A product of K = 128 is 8 steps, each cut once, by 2^-24 of the sum on average, and its two
    operands' terms leave four times that in the mean square (2^-22 at most, 2^-23 on average, each); three products a chunk, over n
    chunks and one more, as independent errors: (3 (8 + 4) (n + 1))^(1/2) 2^-24.  (Cut three times a step, 24 for 8.)"""
    from oracle.deltarule import deltarule_fwd_ref
    from tests.test_gpu_deltarule import _np
    L = 256
    d = _case(2, L, 4, 4, K, V, "f32", decay=False, carry=False, seed=seed)
    o, _, h = _fwd(ss, d)
    ro, rS = deltarule_fwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "beta")])
    tol = (3 * (8 + 4) * (L // 64 + 1)) ** 0.5 * 2.0 ** -24
    for name, got, ref in (("o", o, ro), ("h_last", h, rS[:, -1])):
        off = np.linalg.norm(_np(got) - ref) / np.linalg.norm(ref)
        assert off <= tol, (name, off, tol)
