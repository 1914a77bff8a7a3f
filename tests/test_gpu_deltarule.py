"""The gated delta rule on the GPU against the float64 recurrence.

Tolerance, in the 2-norm of a whole output relative to its own.  A chunk's state comes of three products one after another
(K S0, M (beta R), K^T u), each summed in at most 24 steps of 16 terms; a step is off by at most 2^-23 of the sum so far (the
tensor core's sums are cut, not rounded), the steps' errors add like independent ones, and a cut has one sign, which doubles
them: 2 sqrt(24) 2^-23 a product.  Operands of two fp16 terms (fp32 activations) add 2^-22, less than that.  Keys have length
one and 0 <= beta <= 2, so a token's map of the state is a contraction and what is off is carried on, not amplified: over n
chunks sqrt(n) of it, and one more for the end.  So the forward has F = sqrt(3) 2 sqrt(24) 2^-23 sqrt(n + 1) = 2.1e-6 sqrt(n + 1);
a gradient follows a forward and a backward chain and one more set of products: 3 F.  bf16 outputs have their own rounding too:
eight significant bits, so steps of 2^-7 at a power of two and half of one, 2^-8, at most.  The operands of dq and dk have two bf16
terms, one cut to eight bits and one rounded: 2^-15, which is added twice.
"""

import numpy as np
import pytest

from oracle.deltarule import deltarule_bwd_ref, deltarule_fwd_ref, deltarule_step_ref
from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


def _case(B, L, H, G, K, V, dtype="bf16", decay=True, carry=True, lengths=None, packed=False, strong=False, alike=0.5, seed=0):
    import torch
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cast = lambda a, t=dt: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    unit = lambda a: a / np.linalg.norm(a, axis=-1, keepdims=True)
    d = {"g": None}
    if decay:
        g = -np.exp(r.uniform(np.log(1e-3), np.log(1.0), (B, L, H)))
        if strong:  # now and then nearly all, or all, of the state is forgotten
            at = r.random(g.shape)
            g = np.where(at < 0.05, -np.inf, np.where(at < 0.1, -300.0, np.where(at < 0.15, -30.0, g)))
        d["g"] = cast(g, torch.float32)
    beta = r.uniform(0.0, 2.0, (B, L, H))
    at = r.random(beta.shape)
    d["beta"] = cast(np.where(at < 0.1, 0.0, np.where(at < 0.2, 1.0, beta)), torch.float32)
    q, v = unit(r.standard_normal((B, L, G, K))), r.standard_normal((B, L, H, V))
    k = unit(r.standard_normal((B, L, G, K)) + alike * r.standard_normal((B, 1, G, K)))
    if packed:
        qkv = cast(np.concatenate([a.reshape(B, L, -1) for a in (q, k, v)], -1))
        q, k, v = qkv.split([G * K, G * K, H * V], dim=-1)
        d |= {"q": q.unflatten(-1, (G, K)), "k": k.unflatten(-1, (G, K)), "v": v.unflatten(-1, (H, V))}
    else:
        d |= {"q": cast(q), "k": cast(k), "v": cast(v)}
    d["do"] = cast(r.standard_normal((B, L, H, V)))
    d["h0"] = cast(r.standard_normal((B, H, K, V)), torch.float32) if carry else None
    d["dh_last"] = cast(r.standard_normal((B, H, K, V)), torch.float32) if carry else None
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return d


def _np(t):
    return None if t is None else t.detach().double().cpu().numpy()


def _fwd(ss, d, **kw):
    return ss.deltarule_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], h0=d["h0"], lengths=d["lengths"], **kw)


def _bwd(ss, d, ckpt, **kw):
    return ss.deltarule_bwd(d["q"], d["k"], d["v"], d["g"], d["beta"], ckpt, d["do"], dh_last=d["dh_last"], lengths=d["lengths"], **kw)


def _tol(L, dtype, typed, products):
    f = 3 ** 0.5 * 2 * 24 ** 0.5 * 2.0 ** -23 * (-(-L // 64) + 1) ** 0.5 * products
    return f + (2.0 ** -8 + 2 * 2.0 ** -15 if typed and dtype == "bf16" else 0.0)


def _near(got, ref, tol, name):
    got = _np(got)
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    off, size = np.linalg.norm(got - ref), np.linalg.norm(ref)
    assert off <= tol * size + 1e-30, f"{name}: {off / max(size, 1e-300):.3e} of the norm off, {tol:.3e} allowed"


# B, L, H, G, K, V, options
CASES = [
    (1, 1, 1, 1, 8, 8, {}),
    (2, 3, 2, 1, 16, 24, {"decay": False}),
    (1, 63, 1, 1, 64, 64, {"carry": False}),
    (2, 64, 2, 2, 64, 64, {}),
    (1, 65, 3, 1, 128, 64, {"packed": True}),
    (2, 127, 2, 2, 128, 128, {"alike": 4.0}),
    (1, 128, 2, 1, 128, 128, {"carry": False}),
    (1, 129, 2, 2, 40, 72, {"packed": True}),
    (4, 150, 4, 2, 72, 120, {"lengths": [150, 0, 1, 149]}),
    (6, 130, 2, 1, 24, 128, {"lengths": [128, 129, 64, 0, 130, 65], "decay": False}),
    (2, 200, 2, 1, 64, 96, {"strong": True}),
    (1, 300, 2, 2, 128, 128, {"strong": True, "packed": True}),
    (2, 500, 1, 1, 128, 8, {"lengths": [500, 321]}),
    (1, 700, 3, 1, 8, 128, {"packed": True, "lengths": [640]}),
    (160, 70, 1, 1, 16, 16, {}),  # more walks than SMs
    (3, 90, 5, 5, 56, 40, {"decay": False, "carry": False, "lengths": [-3, 90, 1000]}),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_forward(ss, B, L, H, G, K, V, opt, dtype):
    d = _case(B, L, H, G, K, V, dtype, seed=L + K, **opt)
    o, ckpt, h_last = _fwd(ss, d)
    n = None if d["lengths"] is None else np.clip(_np(d["lengths"]), 0, L)
    ro, rS = deltarule_fwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "beta", "h0")], lengths=n)
    _near(h_last, rS[:, -1], _tol(L, dtype, False, 1), "h_last")
    _near(o, ro, _tol(L, dtype, True, 1), "o")
    o2, none, none2 = _fwd(ss, d, want_ckpt=False, want_h_last=False)
    assert none is None and none2 is None
    _near(o2, ro, _tol(L, dtype, True, 1), "o without checkpoints")
    o3, _, h3 = _fwd(ss, d)
    assert (o3 == o).all() and (h3 == h_last).all()
    assert ss.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_backward(ss, B, L, H, G, K, V, opt, dtype):
    d = _case(B, L, H, G, K, V, dtype, seed=L + V, **opt)
    _, ckpt, _ = _fwd(ss, d)
    got = _bwd(ss, d, ckpt)
    n = None if d["lengths"] is None else np.clip(_np(d["lengths"]), 0, L)
    ref = deltarule_bwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "beta", "do", "h0", "dh_last")], lengths=n)
    for name in ("dh0", "dbeta", "dv", "dq", "dk", "dg"):
        if ref[name] is None:
            assert got[name] is None
            continue
        tol = _tol(L, dtype, name in ("dq", "dk", "dv"), 3)
        if name == "dg":  # a difference of sums over the chunk: what is off is off of them, not of what they leave
            live = np.arange(L)[None, :, None] < (np.full(B, L) if n is None else n)[:, None, None]
            o, S = deltarule_fwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "beta", "h0")], lengths=n)
            terms = np.where(live, np.abs(_np(d["do"]) * o).sum(-1) + np.abs(ref["dv"] * _np(d["v"])).sum(-1), 0.0)
            tol = tol * max(1.0, np.linalg.norm(terms) * 64 ** 0.5 / max(np.linalg.norm(ref["dg"]), 1e-30))
        _near(got[name], ref[name], tol, name)
    again = _bwd(ss, d, ckpt)
    for name, t in got.items():
        assert t is None or (again[name] == t).all(), f"{name}: two identical calls differ"
    assert _bwd(ss, d, ckpt, want_dh0=False)["dh0"] is None
    assert ss.device_status() == 0


def test_gradient_against_differences(ss):
    """Along random directions, fp32: the loss's slope by central differences.  A step s leaves s^2 of a third derivative (the
    loss is a polynomial of low degree in everything but g, and s is small beside one) and the rounding of the two losses, 3 F
    of the terms' norm, over 2 s."""
    import torch
    d = _case(2, 90, 2, 1, 16, 24, "f32", seed=5)
    _, ckpt, _ = _fwd(ss, d)
    grad = _bwd(ss, d, ckpt)

    def loss(a):
        o, _, h = _fwd(ss, a, want_ckpt=False)
        return float((o.double() * d["do"].double()).sum() + (h.double() * d["dh_last"].double()).sum())

    o, _, h = _fwd(ss, d, want_ckpt=False)
    size = float((o * d["do"]).norm() + (h * d["dh_last"]).norm())
    for name in ("q", "k", "v", "g", "beta", "h0"):
        u = torch.randn(d[name].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        u = u / u.norm()
        s = 2.0 ** -5
        slope = (loss(d | {name: d[name] + s * u}) - loss(d | {name: d[name] - s * u})) / (2 * s)
        want = float((grad["d" + name].double() * u.double()).sum())
        total = float(grad["d" + name].double().norm())
        assert abs(slope - want) <= s * s * total + _tol(90, "f32", False, 3) * size / s, (name, slope, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_places_may_hold_anything(ss, dtype):
    """NaN and infinities past a row's length change nothing, and a row of length 0 passes its state through."""
    import torch
    d = _case(5, 200, 2, 1, 64, 64, dtype, lengths=[0, 1, 130, 192, 200], seed=9)
    e = dict(d)
    dead = torch.arange(200, device="cuda")[None, :] >= d["lengths"][:, None]
    for n, x in (("q", "nan"), ("k", "inf"), ("v", "nan"), ("do", "-inf"), ("g", "nan"), ("beta", "inf")):
        m = dead.view(5, 200, *[1] * (d[n].dim() - 2))
        e[n] = torch.where(m, torch.full_like(d[n], float(x)), d[n])
    out = []
    for x in (d, e):
        o, ckpt, h = _fwd(ss, x)
        out.append({"o": o, "h": h, "o2": _fwd(ss, x, want_ckpt=False)[0]} | _bwd(ss, x, ckpt))
    for n in out[0]:
        assert torch.equal(out[0][n], out[1][n]), n
    a = out[1]
    assert torch.equal(a["h"][0], d["h0"][0]) and torch.equal(a["dh0"][0], d["dh_last"][0])
    for n in ("o", "dq", "dk", "dv", "dg", "dbeta"):
        assert (a[n][dead] == 0).all(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", ["q", "k", "v", "g", "beta"])
def test_a_bad_value_stays_in_its_row_and_behind_its_chunk(ss, dtype, where):
    import torch
    d = _case(3, 200, 3, 3, 32, 40, dtype, seed=21)
    o, _, h = _fwd(ss, d)
    for bad in (float("nan"), float("inf")):
        e = dict(d)
        e[where] = d[where].clone()
        e[where][1, 100, 1] = bad
        o2, ckpt, h2 = _fwd(ss, e)
        _bwd(ss, e, ckpt)
        assert torch.equal(o2[0], o[0]) and torch.equal(o2[2], o[2]) and torch.equal(h2[0], h[0]) and torch.equal(h2[2], h[2])
        for head in (0, 2):
            assert torch.equal(o2[1, :, head], o[1, :, head]) and torch.equal(h2[1, head], h[1, head])
        assert torch.equal(o2[1, :64], o[1, :64])
    assert ss.device_status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale_k", [2.0 ** -40, 2.0 ** -6, 2.0 ** 9, 2.0 ** 30])
def test_keys_of_any_length(ss, scale_k, dtype):
    """Keys scaled by a power of two and beta by its square's reciprocal: the state answers scaled keys with the same values, so
    o with queries scaled alike, the states times the scale and the gradients follow exactly what the unit keys give."""
    import torch
    d = _case(2, 150, 2, 1, 48, 40, dtype, seed=4)
    e = d | {"k": d["k"] * scale_k, "beta": d["beta"] * scale_k ** -2, "h0": d["h0"] / scale_k, "q": d["q"] * scale_k,
             "dh_last": d["dh_last"] * scale_k}
    o, ckpt, h = _fwd(ss, d)
    o2, ckpt2, h2 = _fwd(ss, e)
    g, g2 = _bwd(ss, d, ckpt), _bwd(ss, e, ckpt2)
    tol = _tol(150, dtype, False, 3) * 2  # the same arithmetic but for the powers of two a scaled operand takes
    typed = 2.0 ** -7 if dtype == "bf16" else 0.0  # two results that round apart
    for n, a, b, s in (("o", o, o2, 1.0), ("h", h, h2, scale_k), ("dv", g["dv"], g2["dv"], 1.0), ("dk", g["dk"], g2["dk"], scale_k),
                       ("dq", g["dq"], g2["dq"], scale_k), ("dg", g["dg"], g2["dg"], 1.0), ("dbeta", g["dbeta"], g2["dbeta"], scale_k ** -2),
                       ("dh0", g["dh0"], g2["dh0"], scale_k ** -1)):
        t = tol + (typed if n in ("o", "dv", "dk", "dq") else 0.0)
        _near(b.double() * s, _np(a), t, n)


def test_tokens_of_very_different_lengths(ss):
    """Keys of 2^-20 to 2^4 in one chunk: each token's own gradients are right, not only the largest's."""
    r = np.random.default_rng(8)
    for dtype in ("f32", "bf16"):
        d = _case(1, 64, 1, 1, 32, 32, dtype, decay=False, seed=6)
        s = 2.0 ** r.integers(-20, 5, (1, 64, 1, 1))
        import torch
        st = torch.from_numpy(s).cuda()
        d["k"] = (d["k"].double() * st).to(d["k"].dtype)
        d["beta"] = (d["beta"].double() / st[..., 0] ** 2).clamp(max=4.0).float()
        _, ckpt, _ = _fwd(ss, d)
        got = _bwd(ss, d, ckpt)
        ref = deltarule_bwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "beta", "do", "h0", "dh_last")])
        for n in ("dv", "dk", "dq"):
            a, b = _np(got[n])[0, :, 0], ref[n][0, :, 0]
            err = np.linalg.norm(a - b, axis=-1) / np.maximum(np.linalg.norm(b, axis=-1), 1e-30)
            # one token's share of the bounds above: the root of 64 of the whole's
            assert np.all(err <= 8 * _tol(64, dtype, True, 3)), (dtype, n, err.max())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,K,V,decay", [(1, 1, 1, 8, 8, True), (3, 4, 2, 40, 72, False), (2, 32, 32, 128, 128, True),
                                             (300, 2, 1, 64, 128, True), (1, 3, 3, 120, 8, True), (200, 1, 1, 128, 40, False),
                                             (40, 24, 8, 128, 104, True), (520, 1, 1, 64, 64, True), (513, 2, 2, 8, 8, True)])
def test_step(ss, B, H, G, K, V, decay, dtype):
    """Every term of the new state passes two sums of K products in fp32 and five roundings: (2 sqrt(K) + 5) 2^-24 of the norm, and
    o one more sum."""
    d = _case(B, 1, H, G, K, V, dtype, decay=decay, seed=B + K)
    q, k, v, beta = (d[n][:, 0].contiguous() for n in ("q", "k", "v", "beta"))
    g = d["g"][:, 0].contiguous() if decay else None
    h = d["h0"].clone()
    o = ss.deltarule_step(q, k, v, g, beta, h)
    rh, ro = deltarule_step_ref(_np(d["h0"]), _np(q), _np(k), _np(v), _np(g), _np(beta))
    tol = (3 * K ** 0.5 + 8) * 2.0 ** -24
    _near(h, rh, tol, "h")
    _near(o, ro, 2 * tol + (2.0 ** -8 if dtype == "bf16" else 0.0), "o")


def test_prompt_then_steps_equals_one_prompt(ss):
    """fp32: 70 tokens by the chunked form, the next 20 one by one, against 90 by the chunked form."""
    d = _case(2, 90, 4, 2, 64, 64, "f32", seed=11)
    o, _, h = _fwd(ss, d, want_ckpt=False)
    cut = {n: d[n][:, :70].contiguous() for n in ("q", "k", "v", "g", "beta")} | {"h0": d["h0"], "lengths": None}
    _, _, s = _fwd(ss, cut, want_ckpt=False)
    for t in range(70, 90):
        ot = ss.deltarule_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v", "g", "beta")), s)
        _near(ot, _np(o[:, t]), 2 * _tol(90, "f32", False, 1), "o")
    _near(s, _np(h), 2 * _tol(90, "f32", False, 1), "h")


def test_pieces_of_a_sequence(ss):
    """Forward and backward in two pieces, the state handed on and its gradient handed back, against one call."""
    import torch
    d = _case(2, 200, 2, 2, 40, 64, "f32", seed=12)
    _, ckpt, h = _fwd(ss, d)
    g = _bwd(ss, d, ckpt)
    cut = lambda a, b: {n: d[n][:, a:b].contiguous() for n in ("q", "k", "v", "g", "beta", "do")}
    a = cut(0, 75) | {"h0": d["h0"], "lengths": None}
    _, ck_a, h_a = _fwd(ss, a)
    b = cut(75, 200) | {"h0": h_a, "lengths": None, "dh_last": d["dh_last"]}
    _, ck_b, h_b = _fwd(ss, b)
    g_b = _bwd(ss, b, ck_b)
    g_a = _bwd(ss, a | {"dh_last": g_b["dh0"]}, ck_a)
    tol = 2 * _tol(200, "f32", False, 3)
    _near(h_b, _np(h), tol, "h")
    for n in ("dq", "dk", "dv", "dbeta"):
        _near(torch.cat([g_a[n], g_b[n]], 1), _np(g[n]), tol, n)
    _near(g_a["dh0"], _np(g["dh0"]), tol, "dh0")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_on_another_stream_and_from_a_graph(ss, dtype):
    import torch
    d = _case(2, 300, 4, 2, 64, 64, dtype, seed=13)
    o, ckpt, h = _fwd(ss, d)
    g = _bwd(ss, d, ckpt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o2, ckpt2, h2 = _fwd(ss, d)
        g2 = _bwd(ss, d, ckpt2)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(h, h2) and all(torch.equal(g[n], g2[n]) for n in g)
    hs = d["h0"].clone()
    one = [d[n][:, 0].contiguous() for n in ("q", "k", "v", "g", "beta")]
    ss.deltarule_step(*one, hs)
    hs.copy_(d["h0"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, ckpt3, h3 = _fwd(ss, d)
        g3 = _bwd(ss, d, ckpt3)
        os = ss.deltarule_step(*one, hs)
    for n in ("q", "v", "do"):
        d[n].mul_(-0.5)
    d["beta"].mul_(0.5)
    one[2].mul_(3.0)
    hs.copy_(d["h0"])
    graph.replay()
    torch.cuda.synchronize()
    o4, ckpt4, h4 = _fwd(ss, d)
    g4 = _bwd(ss, d, ckpt4)
    assert torch.equal(o3, o4) and torch.equal(h3, h4) and all(torch.equal(g3[n], g4[n]) for n in g3)
    h5 = d["h0"].clone()
    assert torch.equal(os, ss.deltarule_step(*one, h5)) and torch.equal(hs, h5)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_two_calls_at_once(ss, dtype):
    """Two streams, each with its own workspace from the allocator: the same bits as one after the other."""
    import torch
    ds = [_case(2, 200, 8, 8, 64, 64, dtype, seed=s) for s in (1, 2)]
    want = []
    for d in ds:
        o, c, h = _fwd(ss, d)
        want.append((o, h, _bwd(ss, d, c)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    got = [None, None]
    for rep in range(3):
        for i, (d, s) in enumerate(zip(ds, streams)):
            with torch.cuda.stream(s):
                o, c, h = _fwd(ss, d)
                got[i] = (o, h, _bwd(ss, d, c))
        torch.cuda.synchronize()
        for (o, h, g), (o2, h2, g2) in zip(want, got):
            assert torch.equal(o, o2) and torch.equal(h, h2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_workspace_contents_do_not_matter(ss, dtype):
    import torch
    d = _case(2, 150, 4, 2, 72, 40, dtype, lengths=[150, 70], seed=3)
    o, ckpt, h = _fwd(ss, d)
    g = _bwd(ss, d, ckpt)
    for fill in (0xFF, 0x7F):
        ws = torch.full((64 << 20,), fill, dtype=torch.uint8, device="cuda")
        ckpt.view(torch.uint8).fill_(fill)
        o2, ckpt2, h2 = _fwd(ss, d)
        g2 = _bwd(ss, d, ckpt2, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(h, h2) and all(torch.equal(g[n], g2[n]) for n in g)
        ws.fill_(fill)
        o3, _, h3 = _fwd(ss, d, want_ckpt=False, workspace=ws)
        assert torch.equal(h, h3)  # (o differs with and without ckpt in bf16, by its operands' last term)
        ckpt = ckpt2


def test_offsets_past_32_bits(ss):
    """v and o of over 2^31 elements: with strong decays the last tokens see only their neighbours, so they equal a call on the
    tail alone.  A decay of e^-2 a token leaves e^-256 of anything 128 tokens back: nothing in bf16 or fp32."""
    import torch
    L, H, V, K, tail = 270_080, 64, 128, 8, 320
    gen = torch.Generator(device="cuda").manual_seed(1)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    q = unit(torch.randn(1, L, 1, K, device="cuda", generator=gen)).bfloat16()
    k = unit(torch.randn(1, L, 1, K, device="cuda", generator=gen)).bfloat16()
    v = torch.empty(1, L, H, V, device="cuda", dtype=torch.bfloat16)
    v[:, :-tail] = 1.0
    v[:, -tail:] = torch.randn(1, tail, H, V, device="cuda", generator=gen).bfloat16()
    g = torch.full((1, L, H), -2.0, device="cuda")
    beta = torch.rand(1, L, H, device="cuda", generator=gen)
    o, _, h = ss.deltarule_fwd(q, k, v, g, beta, want_ckpt=False)
    cut = lambda t: t[:, -tail:].contiguous()
    o2, _, h2 = ss.deltarule_fwd(cut(q), cut(k), cut(v), cut(g), cut(beta), want_ckpt=False)
    tol = 2 * _tol(tail, "bf16", False, 1)
    _near(o[:, -100:], _np(o2[:, -100:]), 2.0 ** -7 + tol, "o")  # two results that round apart
    _near(h, _np(h2), tol, "h")


@pytest.mark.parametrize("dtype,L,H,V,K,tail", [("bf16", 270_080, 64, 128, 8, 320), ("f32", 65_600, 512, 64, 8, 320)])
def test_gradient_offsets_past_32_bits(ss, dtype, L, H, V, K, tail):
    """As above for the backward: v, do, dv, r and o of over 2^31 elements.  Nothing comes back from the tail, and into its last
    100 tokens comes nothing from before it, so all of their gradients equal those of a call on the tail alone."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(1)
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    assert L * H * V > 2 ** 31
    q, k = (unit(torch.randn(1, L, 1, K, device="cuda", generator=gen)).to(dt) for _ in range(2))
    v, do = (torch.ones(1, L, H, V, device="cuda", dtype=dt) for _ in range(2))
    for t in (v, do):
        t[:, -tail:] = torch.randn(1, tail, H, V, device="cuda", generator=gen).to(dt)
    g = torch.full((1, L, H), -2.0, device="cuda")
    beta = torch.rand(1, L, H, device="cuda", generator=gen)
    _, ckpt, _ = ss.deltarule_fwd(q, k, v, g, beta)
    got = ss.deltarule_bwd(q, k, v, g, beta, ckpt, do, want_dh0=False)
    del ckpt
    cut = lambda t: t[:, -tail:].contiguous()
    c = [cut(t) for t in (q, k, v, g, beta)]
    _, ckpt, _ = ss.deltarule_fwd(*c)
    ref = ss.deltarule_bwd(*c, ckpt, cut(do), want_dh0=False)
    typed = 2.0 ** -7 if dtype == "bf16" else 0.0  # two results that round apart
    for n in ("dq", "dk", "dv", "dg", "dbeta"):
        tol = 2 * _tol(tail, dtype, False, 3) * 64 ** 0.5 + (typed if n in ("dq", "dk", "dv") else 0.0)  # (dg: sums over a chunk)
        _near(got[n][:, -100:], _np(ref[n][:, -100:]), tol, n)


def test_refusals(ss):
    import torch
    z = lambda *s: torch.zeros(*s, device="cuda")
    q, v, g = z(2, 4, 2, 16), z(2, 4, 4, 16), z(2, 4, 4)
    with pytest.raises(ValueError, match="shape"):
        ss.deltarule_fwd(q, q[:, :3], v, g, g)
    with pytest.raises(ValueError, match="beta has shape"):
        ss.deltarule_fwd(q, q, v, g, g[:, :, :2].contiguous())
    with pytest.raises(ValueError, match="float32"):
        ss.deltarule_fwd(q, q, v, g.double(), g)
    with pytest.raises(ValueError, match="torch.float32, got torch.bfloat16"):
        ss.deltarule_fwd(q, q, v.bfloat16(), g, g)
    with pytest.raises(ValueError, match="strides"):
        ss.deltarule_fwd(q[..., ::2], q[..., ::2], v, g, g)
    with pytest.raises(ValueError, match="lengths"):
        ss.deltarule_fwd(q, q, v, g, g, lengths=z(2))
    with pytest.raises(ss.SSError, match="status -4"):
        ss.deltarule_fwd(q[..., :4].contiguous(), q[..., :4].contiguous(), v, g, g)
    with pytest.raises(ss.SSError, match="status -2"):
        ss.deltarule_fwd(z(2, 4, 3, 16), z(2, 4, 3, 16), v, g, g)
    with pytest.raises(ss.SSError, match="status -1"):  # an empty tensor has no memory
        ss.deltarule_fwd(q[:, :0], q[:, :0], v[:, :0], g[:, :0], g[:, :0])
    with pytest.raises(ValueError, match="ckpt"):
        ss.deltarule_bwd(q, q, v, g, g, z(1), v)
    with pytest.raises(ss.SSError, match="status -5"):
        ss.deltarule_fwd(q, q, v, g, g, want_ckpt=False, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="h has shape"):
        ss.deltarule_step(q[:, 0].contiguous(), q[:, 0].contiguous(), v[:, 0].contiguous(), None, g[:, 0].contiguous(), z(2, 4, 16, 8))
