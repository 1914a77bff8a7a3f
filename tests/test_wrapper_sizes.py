"""Sizes that do not fit the library's 32-bit integers are refused before anything is allocated or launched (CPU: tensors are known by
their shapes alone)."""

import pytest

torch = pytest.importorskip("torch")
from tests.test_deltarule_wrappers import _as, _on, ops  # noqa: E402,F401  (the stand-in library)

EMPTY = torch.empty  # (the stand-in makes outputs in host memory)
BIG = (1 << 31) + 64  # cut to 32 bits: 64


def _shape(*shape, dtype=torch.bfloat16):
    return _as(EMPTY(shape, dtype=dtype, device="meta"), 0)


def test_delta_rule_and_linear_attention(ops):  # noqa: F811
    mod, lib = ops
    f = torch.float32
    for B, L in ((1, BIG), (BIG, 1)):
        q, v, g = _shape(B, L, 1, 8), _shape(B, L, 1, 8), _shape(B, L, 1, dtype=f)
        for call in (lambda: mod.deltarule_fwd(q, q, v, g, g), lambda: mod.deltarule_fwd(q, q, v, g, g, want_ckpt=False),
                     lambda: mod.deltarule_bwd(q, q, v, g, g, _on(0, 1), v), lambda: mod.linattn_fwd(q, q, v, g),
                     lambda: mod.linattn_bwd(q, q, v, g, _on(0, 1), v)):
            with pytest.raises(ValueError, match="2\\^31"):
                call()
    assert not lib.launched


@pytest.mark.parametrize("shape", [(BIG, 8), (BIG, 1, 8), (1, BIG, 8), (2, 1 << 16, (1 << 15) + 1, 8)])
def test_group_norm(ops, shape):  # noqa: F811
    mod, lib = ops
    x, w, st = _shape(*shape), _on(0, 8), _on(0, 1)
    with pytest.raises(ValueError, match="2\\^31"):
        mod.groupnorm_fwd(x, w, w, 1, 1e-5)
    with pytest.raises(ValueError, match="2\\^31"):
        mod.groupnorm_bwd(x, x, w, w, st, st, 1)
    assert not lib.launched


@pytest.mark.parametrize("shape", [(BIG, 8), (1, BIG, 8), (BIG, 1, 8)])
def test_the_other_calls(ops, shape):  # noqa: F811
    mod, lib = ops
    x, w = _shape(*shape), _on(0, 8)
    calls = [lambda: mod.layernorm_fwd(x, w, w, 1e-5), lambda: mod.rmsnorm_fwd(x, w, 1e-5), lambda: mod.layernorm_bwd(x, x, w, w, w),
             lambda: mod.rmsnorm_bwd(x, x, w, w)] if len(shape) == 2 else [
        lambda: mod.ss_scan_fwd(x, x, _on(0, 8, 4), x, x, w, x), lambda: mod.conv1d_causal_fwd(x, _on(0, 8, 4)),
        lambda: mod.conv1d_causal_bwd(x, x, _on(0, 8, 4))]
    for call in calls:
        with pytest.raises(ValueError, match="2\\^31"):
            call()
    assert not lib.launched
