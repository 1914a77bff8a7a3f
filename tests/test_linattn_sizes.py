"""Sizes of linear attention whose products or chunks pass an int: the status before anything is launched (CPU)."""

import ctypes
import os
import shutil

import pytest


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    from mamba_selective_ssm_gb300 import _build, _capi
    _build.build()
    return _capi.load()


P = [ctypes.c_void_p(0x100000 + 4096 * i) for i in range(14)]


def _fwd(lib, dtype, ld, B, L, H, G, K, V):
    return lib.linattn_fwd(P[0], ld[0], P[1], ld[1], P[2], ld[2], P[3], 0, P[4], None, P[6], P[7], P[8], B, L, H, G, K, V, 0.1, dtype,
                           None, 0, None)


def _bwd(lib, dtype, ld, B, L, H, G, K, V):
    return lib.linattn_bwd(P[0], ld[0], P[1], ld[1], P[2], ld[2], P[3], 0, None, *P[5:13], B, L, H, G, K, V, 0.1, dtype, None, 0,
                           None)


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_a_stride_below_a_token_of_2_to_the_31_elements(lib, call, dtype):
    """heads * width is 2^31: a stride of one head's width is not a token's."""
    from mamba_selective_ssm_gb300 import _capi as c
    n = 1 << 24
    assert call(lib, dtype, (n * 128, 8, n * 8), 1, 1, n, n, 128, 8) == c.SS_ERR_DIM
    assert call(lib, dtype, (8, n * 128, n * 8), 1, 1, n, n, 128, 8) == c.SS_ERR_DIM
    assert call(lib, dtype, (8, 8, 8), 1, 1, n, 1, 8, 128) == c.SS_ERR_DIM


@pytest.mark.parametrize("L", [2147483137, 2147483647])
def test_rows_near_the_largest_int(lib, L):
    from mamba_selective_ssm_gb300 import _capi as c
    for dtype in (0, 1):
        assert lib.linattn_num_chunks(L, dtype) == 0
        assert lib.linattn_fwd_workspace_size(1, L, 1, 1, 8, 8, dtype) == 0
        assert lib.linattn_bwd_workspace_size(1, L, 1, 1, 8, 8, 0, dtype) == 0
        assert _fwd(lib, dtype, (8, 8, 8), 1, L, 1, 1, 8, 8) == c.SS_ERR_DIM
        assert _bwd(lib, dtype, (8, 8, 8), 1, L, 1, 1, 8, 8) == c.SS_ERR_DIM


def test_the_longest_row_has_its_chunks(lib):
    L = 2147483136
    assert lib.linattn_num_chunks(L, 0) == L // 64 and lib.linattn_num_chunks(L, 1) == L // 128
    assert lib.linattn_fwd_workspace_size(1, L, 1, 1, 8, 8, 1) > 0
