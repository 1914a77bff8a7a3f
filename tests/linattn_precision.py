"""How far linear attention's outputs may be from the float64 recurrence in the root mean square, and one chunk of it
restated in float64 with its operands rounded as told (what the bounds let pass and what they do not is tested on that).

The worst-case bounds of test_gpu_linattn.py count every step at its largest and in one direction; rounding errors of
many terms do not add up like that, and a lost term hides below them.  In the root mean square:

* bf16 activations, outputs of that type (o, dq, dk, dv): an operand (a score or a state) is rounded to bf16 once and the
  output once.  Independent roundings of one size add up to sqrt(2) of one; the size is that of the reference's own
  rounding to bf16.  A quarter is added for operands whose values lie less well within their binades.
* bf16 activations, fp32 outputs (h_last, dg, dh0): operands are three bf16 terms, 2^-24 of the value, so that what counts are
  sums and exponentials.  The tensor core cuts a sum instead of rounding it, by 2^-24 on average; at most 16 of the
  cut sums are about as large as the result (eight steps of 16 for the first term, eight for a term added after it).
  Two exponentials of the hardware, 2^-22 each, and a rounding: 16 + 2 * 4 + 1 = 25 times 2^-24 = 1.5e-6.
  (Operands in two terms: a rounding of what the first leaves, (2^-7 / sqrt(12) / 1.5)^2 = 2.3e-6.)
* fp32 activations: products of operands of 22 bits, at most three one after another, each off by 2^-22 with the sums'
  cuts and the decays: 2^-19 leaves a factor of two.  (An operand in one tf32 value, 11 bits: 2e-4; in 16 bits: 6e-6.)
"""

import numpy as np

FP32_OF_BF16 = 25 * 2.0 ** -24
FP32 = 2.0 ** -19


def bits(x, n):
    """x rounded to n significant bits, to nearest."""
    m, e = np.frexp(np.asarray(x, np.float64))
    return np.ldexp(np.rint(m * 2.0 ** n) / 2.0 ** n, e)


def terms(x, n):
    """x as the sum of n bf16 terms."""
    left, s = np.asarray(x, np.float64), 0.0
    for _ in range(n):
        t = bits(left, 8)
        s, left = s + t, left - t
    return s


def rms(x):
    return float(np.sqrt(np.mean(np.square(x))))


def off(got, ref):
    return rms(got - ref) / rms(ref)


def bound(name, ref, dtype):
    if dtype == "f32":
        return FP32
    if name in ("o", "dq", "dk", "dv"):
        return 1.25 * 2 ** 0.5 * off(bits(ref, 8), ref)
    return FP32_OF_BF16


CASES = {  # which operands an output is made of: scale of the first state, of the last state's gradient
    "scores": (0.0, 0.0),
    "state in": (16.0, 0.0),
    "state out": (0.0, 16.0),
}


def inputs(case, B, L, H, G, K, V, seed):
    """float64 arrays whose q, k, v, do are bf16 values and whose g, h0, dh_last are fp32 values."""
    r = np.random.default_rng(seed)
    h, u = CASES[case]
    half = lambda *s: bits(r.standard_normal(s), 8)
    full = lambda *s: r.standard_normal(s).astype(np.float32).astype(np.float64)
    return {"q": half(B, L, G, K), "k": half(B, L, G, K), "v": half(B, L, H, V), "do": half(B, L, H, V),
            "g": (-np.exp(r.uniform(np.log(1e-3), np.log(1e-2), (B, L, H)))).astype(np.float32).astype(np.float64),
            "h0": h * full(B, H, K, V), "dh_last": u * full(B, H, K, V)}


def chunk(d, score=8, state=8, split=3, typed=8):
    """One chunk forward and backward.  Scores and the states that make o and dv rounded to `score` and `state` bits, the other
    fp32 operands as `split` bf16 terms (0: exact), typed outputs rounded to `typed` bits."""
    B, L, G, K = d["q"].shape
    H, V = d["v"].shape[2:]
    sc = K ** -0.5
    part = (lambda x: terms(x, split)) if split else (lambda x: x)
    rep = lambda x: np.repeat(x, H // G, 2).transpose(0, 2, 1, 3)  # [B, H, L, K]
    q, k, v, do = rep(d["q"]), rep(d["k"]), d["v"].transpose(0, 2, 1, 3), d["do"].transpose(0, 2, 1, 3)
    c = np.cumsum(d["g"], 1).transpose(0, 2, 1)
    into, rest, last = np.exp(c)[..., None], np.exp(c[..., -1:] - c)[..., None], np.exp(c[..., -1])[..., None, None]
    S, U = d["h0"], d["dh_last"]
    T = lambda x: x.swapaxes(-1, -2)
    low = np.tril(np.ones((L, L), bool))
    D = np.where(low, np.exp(np.where(low, c[..., :, None] - c[..., None, :], 0.0)), 0.0) * sc
    P, dP = (q @ T(k)) * D, (do @ T(v)) * D
    rP, rdP = bits(P, score), bits(dP, score)
    o = rP @ v + sc * into * (q @ bits(S, state))
    qi, ki = sc * into * (do @ T(part(S))), rest * (v @ T(part(U)))
    dq, dk = rdP @ k + qi, T(rdP) @ q + ki
    dv = T(rP) @ do + rest * (k @ bits(U, state))
    M = P * (do @ T(v))
    a, b = (q * qi).sum(-1), (k * ki).sum(-1)
    rect = np.where(low, np.cumsum(M, -1) - M, 0.0).sum(-2)
    dg = rect + np.cumsum(a[..., ::-1], -1)[..., ::-1] + np.cumsum(b, -1) - b + (last * S * U).sum((-1, -2))[..., None]
    tok = lambda x: bits(x.transpose(0, 2, 1, 3), typed)
    share = lambda x: bits(x.transpose(0, 2, 1, 3).reshape(B, L, G, H // G, K).sum(3), typed)
    return {"o": tok(o), "h_last": last * S + T(k) @ part(rest * v), "dq": share(dq), "dk": share(dk), "dv": tok(dv),
            "dg": dg.transpose(0, 2, 1), "dh0": last * U + T(q) @ part(sc * into * do)}
