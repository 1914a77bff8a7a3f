"""Linear attention with a decay for each head on the GPU against the float64 recurrence.

Tolerance, element by element: with A the same sum taken over absolute values, every term of an output passes
  - fp32 steps only: at most K + V + 3 * 128 additions or products of a chunk, and one decay of its state per
    chunk (4 half-steps of fp32 for the hardware's exp2 and the product), each off by at most 2^-23 of A
    (one step, twice the half-step: the tensor core's sums are cut, not rounded);
  - with bf16 activations also one rounding of a score or of a state to bf16 (2^-8 of A) and the output's own (2^-8
    of the value).
"""

import numpy as np
import pytest

from oracle.linattn import linattn_bwd_ref, linattn_fwd_ref, linattn_step_ref
from tests.gpu_util import ss_module

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ss():
    return ss_module()


def _case(B, L, H, G, K, V, dtype="bf16", per_head=False, carry=True, lengths=None, packed=False, strong=False, seed=0):
    import torch
    r = np.random.default_rng(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    cast = lambda a, t=dt: torch.from_numpy(np.ascontiguousarray(a)).to(t).cuda()
    g = -np.exp(r.uniform(np.log(1e-3), np.log(1.0), (H,) if per_head else (B, L, H)))
    if strong:  # now and then nearly all, or all, of the state is forgotten
        at = r.random(g.shape)
        g = np.where(at < 0.05, -np.inf, np.where(at < 0.1, -300.0, np.where(at < 0.15, -30.0, g)))
    d = {"g": cast(g, torch.float32)}
    if packed:
        qkv = cast(r.standard_normal((B, L, 2 * G * K + H * V)))
        q, k, v = qkv.split([G * K, G * K, H * V], dim=-1)
        d |= {"q": q.unflatten(-1, (G, K)), "k": k.unflatten(-1, (G, K)), "v": v.unflatten(-1, (H, V))}
    else:
        d |= {"q": cast(r.standard_normal((B, L, G, K))), "k": cast(r.standard_normal((B, L, G, K))),
              "v": cast(r.standard_normal((B, L, H, V)))}
    d["do"] = cast(r.standard_normal((B, L, H, V)))
    d["h0"] = cast(r.standard_normal((B, H, K, V)), torch.float32) if carry else None
    d["dh_last"] = cast(r.standard_normal((B, H, K, V)), torch.float32) if carry else None
    d["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    return d


def _np(t, absolute=False):
    if t is None:
        return None
    a = t.detach().double().cpu().numpy()
    return np.abs(a) if absolute else a


def _close(got, ref, bound, dims, dtype, typed, name):
    K, V, chunks = dims
    got = _np(got)
    tol = 2.0 ** -23 * (K + V + 3 * 128 + 4 * chunks) * bound
    if typed and dtype == "bf16":
        tol = tol + 2.0 ** -8 * (np.abs(ref) + 1.01 * bound)
    assert got.shape == ref.shape, name
    assert np.all(np.isfinite(got)), f"{name}: non-finite values"
    over = np.abs(got - ref) - tol
    assert np.all(over <= 1e-30), f"{name}: {np.abs(got - ref).max():.3e} off, {np.sum(over > 1e-30)} over the bound"


def _forward(d):
    args = [_np(d[n]) for n in ("q", "k", "v")]
    n = _np(d["lengths"])
    o, S = linattn_fwd_ref(*args, _np(d["g"]), _np(d["h0"]), lengths=n)
    ao, aS = linattn_fwd_ref(*[np.abs(a) for a in args], _np(d["g"]), _np(d["h0"], True), lengths=n)
    return o, S[:, -1], ao, aS[:, -1]


def _backward(d):
    n = _np(d["lengths"])
    ref = linattn_bwd_ref(*[_np(d[x]) for x in ("q", "k", "v", "g", "do", "h0", "dh_last")], lengths=n)
    bound = linattn_bwd_ref(_np(d["q"], True), _np(d["k"], True), _np(d["v"], True), _np(d["g"]), _np(d["do"], True), _np(d["h0"], True),
                            _np(d["dh_last"], True), lengths=n)
    return ref, bound


# B, L, H, G, K, V, options
CASES = [
    (1, 1, 1, 1, 8, 8, {}),
    (2, 3, 2, 1, 16, 24, {"per_head": True}),
    (1, 63, 1, 1, 64, 64, {"carry": False}),
    (2, 64, 2, 2, 64, 64, {}),
    (1, 65, 3, 1, 128, 64, {"packed": True}),
    (2, 127, 2, 2, 128, 128, {}),
    (1, 128, 2, 1, 128, 128, {"carry": False}),
    (1, 129, 2, 2, 40, 72, {"packed": True}),
    (4, 150, 4, 2, 72, 120, {"lengths": [150, 0, 1, 149]}),
    (5, 130, 2, 1, 24, 128, {"lengths": [128, 129, 64, 0, 130], "per_head": True}),
    (2, 200, 2, 1, 64, 96, {"strong": True}),
    (1, 300, 2, 2, 128, 128, {"strong": True, "packed": True}),
    (1, 1100, 2, 1, 32, 16, {}),  # cut in segments
    (2, 1024, 1, 1, 128, 64, {"lengths": [1024, 700]}),
    (1, 1500, 3, 1, 64, 128, {"per_head": True, "packed": True, "lengths": [1400]}),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_forward(ss, B, L, H, G, K, V, opt, dtype):
    d = _case(B, L, H, G, K, V, dtype, seed=L + K, **opt)
    o, ckpt, h_last = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], lengths=d["lengths"])
    ro, rS, bo, bS = _forward(d)
    dims = (K, V, ckpt.shape[2])
    _close(h_last, rS, bS, dims, dtype, False, "h_last")
    _close(o, ro, bo, dims, dtype, True, "o")
    o2, none, none2 = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], lengths=d["lengths"], want_ckpt=False,
                                     want_h_last=False)
    assert none is None and none2 is None and (o2 == o).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,H,G,K,V,opt", CASES)
def test_backward(ss, B, L, H, G, K, V, opt, dtype):
    d = _case(B, L, H, G, K, V, dtype, seed=L + V, **opt)
    _, ckpt, _ = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], lengths=d["lengths"])
    got = ss.linattn_bwd(d["q"], d["k"], d["v"], d["g"], ckpt, d["do"], dh_last=d["dh_last"], lengths=d["lengths"])
    ref, bound = _backward(d)
    dims = (K, V, ckpt.shape[2])
    for name in ("dh0", "dg", "dv", "dq", "dk"):
        _close(got[name], ref[name], bound[name], dims, dtype, name in ("dq", "dk", "dv"), name)
    again = ss.linattn_bwd(d["q"], d["k"], d["v"], d["g"], ckpt, d["do"], dh_last=d["dh_last"], lengths=d["lengths"])
    for name, t in got.items():
        assert (again[name] == t).all(), f"{name}: two identical calls differ"


def test_gradient_against_differences(ss):
    """Along random directions, fp32: the loss's slope by central differences.  A step s gives the slope to
    s^2 times a third derivative (the loss is trilinear in q, k, v: exact; analytic in g) plus the rounding of the two
    losses, 2^-22 of the sum of absolute terms, over 2 s."""
    import torch
    d = _case(2, 90, 2, 1, 16, 24, "f32", seed=5)
    _, ckpt, _ = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"])
    grad = ss.linattn_bwd(d["q"], d["k"], d["v"], d["g"], ckpt, d["do"], dh_last=d["dh_last"])

    def loss(a):
        o, _, h = ss.linattn_fwd(a["q"], a["k"], a["v"], a["g"], h0=a["h0"], want_ckpt=False)
        return float((o.double() * d["do"].double()).sum() + (h.double() * d["dh_last"].double()).sum())

    o, _, h = ss.linattn_fwd(*[d[n].abs() for n in ("q", "k", "v")], d["g"], h0=d["h0"].abs(), want_ckpt=False)
    size = float((o * d["do"].abs()).sum() + (h * d["dh_last"].abs()).sum())
    for name in ("q", "k", "v", "g", "h0"):
        u = torch.randn(d[name].shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
        if name == "g":
            u = u * 0.1
        s = 2.0 ** -6
        slope = (loss(d | {name: d[name] + s * u}) - loss(d | {name: d[name] - s * u})) / (2 * s)
        want = float((grad["d" + name].double() * u.double()).sum())
        tol = 2.0 ** -22 * size / s + (s * s * size if name == "g" else 0.0)
        assert abs(slope - want) <= tol, (name, slope, want, tol)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_masked_places_may_hold_anything(ss, dtype):
    """NaN and infinities past a row's length change nothing, and a row of length 0 passes its state through."""
    import torch
    d = _case(4, 200, 2, 1, 64, 64, dtype, lengths=[0, 1, 130, 200], seed=9)
    e = dict(d)
    dead = torch.arange(200, device="cuda")[None, :] >= d["lengths"][:, None]
    for n, x in (("q", float("nan")), ("k", float("inf")), ("v", float("nan")), ("do", float("-inf")), ("g", float("nan"))):
        m = dead.view(4, 200, *[1] * (d[n].dim() - 2))
        e[n] = torch.where(m, torch.full_like(d[n], x), d[n])
    out = []
    for x in (d, e):
        o, ckpt, h = ss.linattn_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], lengths=x["lengths"])
        g = ss.linattn_bwd(x["q"], x["k"], x["v"], x["g"], ckpt, x["do"], dh_last=x["dh_last"], lengths=x["lengths"])
        out.append({"o": o, "h": h} | g)
    for n in out[0]:
        assert torch.equal(out[0][n], out[1][n]), n
    a = out[1]
    assert torch.equal(a["h"][0], d["h0"][0]) and torch.equal(a["dh0"][0], d["dh_last"][0])
    for n in ("o", "dq", "dk", "dv", "dg"):
        assert (a[n][dead] == 0).all(), n


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,H,G,K,V,per_head", [(1, 1, 1, 8, 8, False), (3, 4, 2, 40, 72, True), (2, 32, 32, 128, 128, False),
                                                (300, 2, 1, 64, 128, False), (1, 3, 3, 120, 8, True)])
def test_step(ss, B, H, G, K, V, per_head, dtype):
    d = _case(B, 1, H, G, K, V, dtype, per_head=per_head, seed=B + K)
    q, k, v = (d[n][:, 0].contiguous() for n in "qkv")
    g = d["g"] if per_head else d["g"][:, 0].contiguous()
    h = d["h0"].clone()
    o = ss.linattn_step(q, k, v, g, h)
    rh, ro = linattn_step_ref(_np(d["h0"]), _np(q), _np(k), _np(v), _np(g))
    bh, bo = linattn_step_ref(_np(d["h0"], True), _np(q, True), _np(k, True), _np(v, True), _np(g))
    assert np.all(np.abs(_np(h) - rh) <= 4 * 2.0 ** -23 * bh)  # a decay, two products and a sum
    _close(o, ro, bo, (K, V, 0), dtype, True, "o")


def test_prompt_then_steps_equals_one_prompt(ss):
    """fp32: 70 tokens by the chunked form, the next 20 one by one, against 90 by the chunked form."""
    d = _case(2, 90, 4, 2, 64, 64, "f32", seed=11)
    o, _, h = ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"], want_ckpt=False)
    cut = lambda n, a, b: d[n][:, a:b].contiguous()
    _, _, s = ss.linattn_fwd(cut("q", 0, 70), cut("k", 0, 70), cut("v", 0, 70), cut("g", 0, 70), h0=d["h0"], want_ckpt=False)
    _, _, bo, bS = _forward(d)
    for t in range(70, 90):
        ot = ss.linattn_step(*(d[n][:, t].contiguous() for n in ("q", "k", "v", "g")), s)
        _close(ot, _np(o[:, t]), bo[:, t], (64, 64, 2), "f32", True, "o")
    _close(s, _np(h), bS, (64, 64, 2), "f32", False, "h")


def test_on_another_stream_and_from_a_graph(ss):
    import torch
    d = _case(2, 1100, 2, 1, 64, 64, "bf16", seed=13)
    call = lambda: ss.linattn_fwd(d["q"], d["k"], d["v"], d["g"], h0=d["h0"])
    back = lambda ckpt: ss.linattn_bwd(d["q"], d["k"], d["v"], d["g"], ckpt, d["do"], dh_last=d["dh_last"])
    o, ckpt, h = call()
    g = back(ckpt)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o2, ckpt2, h2 = call()
        g2 = back(ckpt2)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(h, h2) and all(torch.equal(g[n], g2[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o3, ckpt3, h3 = call()
        g3 = back(ckpt3)
    for n in ("q", "k", "v", "do"):
        d[n].mul_(-1.0)  # o, dq, dk, dv change sign with three of the four
    graph.replay()
    torch.cuda.synchronize()
    o4, ckpt4, h4 = call()
    g4 = back(ckpt4)
    assert torch.equal(o3, o4) and torch.equal(h3, h4) and all(torch.equal(g3[n], g4[n]) for n in g3)


def test_offsets_past_32_bits(ss):
    """v and o of over 2^31 elements: with strong decays the last tokens see only their neighbours, so they equal a call on
    the tail alone.  A decay of e^-2 a token leaves e^-256 of anything 128 tokens back: nothing in bf16 or fp32."""
    import torch
    L, H, V, K, tail = 270_080, 64, 128, 8, 320
    gen = torch.Generator(device="cuda").manual_seed(1)
    q = torch.randn(1, L, 1, K, device="cuda", generator=gen).bfloat16()
    k = torch.randn(1, L, 1, K, device="cuda", generator=gen).bfloat16()
    v = torch.empty(1, L, H, V, device="cuda", dtype=torch.bfloat16)
    v[:, :-tail] = 1.0
    v[:, -tail:] = torch.randn(1, tail, H, V, device="cuda", generator=gen).bfloat16()
    g = torch.full((H,), -2.0, device="cuda")
    o, _, h = ss.linattn_fwd(q, k, v, g, want_ckpt=False)
    cut = lambda t: t[:, -tail:].contiguous()
    o2, _, h2 = ss.linattn_fwd(cut(q), cut(k), cut(v), g, want_ckpt=False)
    got, want = o[:, -100:].float(), o2[:, -100:].float()
    size = want.abs().max()
    assert (got - want).abs().max() <= 2.0 ** -6 * size  # chunk borders lie elsewhere: two roundings each, of terms up to the largest
    assert (h - h2).abs().max() <= 2.0 ** -18 * h2.abs().max()


def test_refusals(ss):
    import torch
    q, v, g = torch.zeros(2, 4, 2, 16, device="cuda"), torch.zeros(2, 4, 4, 16, device="cuda"), torch.zeros(2, 4, 4, device="cuda")
    with pytest.raises(ValueError, match="shape"):
        ss.linattn_fwd(q, q[:, :3], v, g)
    with pytest.raises(ValueError, match="float32"):
        ss.linattn_fwd(q, q, v, g.double())
    with pytest.raises(ValueError, match="torch.float32, got torch.bfloat16"):
        ss.linattn_fwd(q, q, v.bfloat16(), g)
    with pytest.raises(ValueError, match="strides"):
        ss.linattn_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), q, v, g)
    with pytest.raises(ValueError, match="strides"):
        ss.linattn_fwd(q[..., ::2], q[..., ::2], v, g)
    with pytest.raises(ValueError, match="lengths"):
        ss.linattn_fwd(q, q, v, g, lengths=torch.zeros(2, device="cuda"))
    with pytest.raises(ss.SSError, match="status -4"):
        ss.linattn_fwd(q[..., :4].contiguous(), q[..., :4].contiguous(), v, g)
    with pytest.raises(ss.SSError, match="status -2"):
        ss.linattn_fwd(torch.zeros(2, 4, 3, 16, device="cuda"), torch.zeros(2, 4, 3, 16, device="cuda"), v, g)
    with pytest.raises(ss.SSError, match="status -1"):  # an empty tensor has no memory
        ss.linattn_fwd(q[:, :0], q[:, :0], v[:, :0], g[:, :0])
    with pytest.raises(ValueError, match="ckpt"):
        ss.linattn_bwd(q, q, v, g, torch.zeros(1, device="cuda"), v)
    with pytest.raises(ValueError, match="h has shape"):
        ss.linattn_step(q[:, 0].contiguous(), q[:, 0].contiguous(), v[:, 0].contiguous(), g[:, 0].contiguous(), torch.zeros(2, 4, 16, 8, device="cuda"))
