"""The root-mean-square bounds of linear attention: a chunk restated with the kernels' roundings keeps them, one whose
scores or states are a bit coarser or whose operands lose a term does not (CPU)."""

import numpy as np
import pytest

from oracle.linattn import linattn_bwd_ref, linattn_fwd_ref
from tests.linattn_precision import CASES, bound, chunk, inputs, off

SHAPE = (2, 128, 4, 2)
HEADS = [(64, 64), (128, 128), (72, 120), (128, 64)]


@pytest.fixture(scope="module", params=[(c, K, V) for c in CASES for K, V in HEADS], ids=lambda p: f"{p[0]}-{p[1]}x{p[2]}")
def case(request):
    name, K, V = request.param
    d = inputs(name, *SHAPE, K, V, seed=K + V)
    o, S = linattn_fwd_ref(*(d[n] for n in ("q", "k", "v", "g", "h0")))
    ref = {"o": o, "h_last": S[:, -1]} | linattn_bwd_ref(*(d[n] for n in ("q", "k", "v", "g", "do", "h0", "dh_last")))
    return name, d, ref


def test_restated_chunk_is_the_recurrence(case):
    _, d, ref = case
    got = chunk(d, score=60, state=60, split=0, typed=60)
    for n, r in ref.items():
        np.testing.assert_allclose(got[n], r, rtol=0, atol=1e-12 * np.abs(r).max(), err_msg=n)


def test_the_kernels_roundings_keep_the_bounds(case):
    _, d, ref = case
    got = chunk(d)
    for n, r in ref.items():
        assert off(got[n], r) <= 0.9 * bound(n, r, "bf16"), n
    got = chunk(d, score=22, state=22, split=0, typed=24)
    for n, r in ref.items():
        assert off(got[n], r) <= 0.5 * bound(n, r, "f32"), n


def _over(case, names, dtype, **roundings):
    _, d, ref = case
    got = chunk(d, **roundings)
    for n in names:
        assert off(got[n], ref[n]) > bound(n, ref[n], dtype), (n, off(got[n], ref[n]), bound(n, ref[n], dtype))


def test_coarser_operands_do_not(case):
    scores, states = {"scores": (("o", "dq", "dk", "dv"), ()), "state in": ((), ("o",)), "state out": ((), ("dv",))}[case[0]]
    _over(case, scores, "bf16", score=7)
    _over(case, states, "bf16", state=7)
    _over(case, scores, "f32", score=16, state=24, split=0, typed=24)
    _over(case, states, "f32", score=24, state=16, split=0, typed=24)


def test_a_lost_term_does_not(case):
    names = {"scores": ("h_last", "dh0"), "state in": ("dg",), "state out": ("dg",)}[case[0]]
    _over(case, names, "bf16", split=2)
