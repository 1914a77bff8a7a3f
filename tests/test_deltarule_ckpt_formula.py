"""The size of a gated delta rule checkpoint as the header states it (CPU)."""

import os
import re
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


def test_checkpoint_sizes_are_the_headers(lib):
    text = open(os.path.join(ROOT, "include", "ssscan.h")).read()
    forms = dict((t, f) for f, t in re.findall(r"\*\s+(\(n \+ 1\) K V \+ 128 n V \+ n \([0-9 +]+\))\s+(fp32|bf16)", text))
    assert sorted(forms) == ["bf16", "fp32"]
    for dtype, name in ((0, "fp32"), (1, "bf16")):
        form = forms[name].replace(") K V", ") * K * V").replace("128 n V", "128 * n * V").replace("n (", "n * (")
        for L, K, V in ((1, 8, 8), (64, 32, 40), (65, 128, 128), (2048, 64, 72), (16384, 128, 64)):
            assert lib.deltarule_ckpt_size(L, K, V, dtype) == eval(form, {"n": -(-L // 64), "K": K, "V": V})
