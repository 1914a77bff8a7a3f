"""Group norm's widest samples, and that every case the measured ranges can draw is within the operators' limits (CPU)."""

import importlib.util
import os
import random
import shutil

import pytest

from tests.conftest import ROOT


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from mamba_selective_ssm_gb300 import _build, _capi
    _build.build()
    return _capi.load()


def test_widest_samples(lib):
    size = lambda C, groups: lib.groupnorm_bwd_workspace_size(2, 3, C, groups, 0)  # noqa: E731
    assert size(32768, 1) and size(32768, 32768) and size(1 << 20, 1 << 12) and size(259080, 1016)
    assert not size(32776, 8) and not size((1 << 20) + 256, (1 << 12) + 1) and not size(65536, 128)


def test_drawn_cases_are_taken(lib):
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    rng = random.Random(5)
    widest = 0
    for c in mod.listed() + [mod.draw(rng) for _ in range(20000)]:
        dt = 1 if c["dtype"] == "bf16" else 0
        if c["op"].startswith("norm"):
            assert lib.groupnorm_bwd_workspace_size(c["N"], c["M"], c["C"], c["groups"], dt) > 0, c
            widest = max(widest, c["C"])
        else:
            sizes = [c[n] for n in "BLHGKV"]
            assert lib.deltarule_fwd_workspace_size(*sizes, dt) > 0 and lib.deltarule_bwd_workspace_size(*sizes, dt) > 0, c
    assert widest > 32768
