"""Refusals of the gated delta rule's and group norm's entry points: the documented status before anything is launched
(CPU)."""

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


def _fake(addr):
    return ctypes.c_void_p(addr)


P = [_fake(0x100000 + 4096 * i) for i in range(16)]
WS = _fake(0x900000)
INT_MAX = 2147483647


def _sizes(**kw):
    s = dict(B=2, L=100, H=4, G=2, K=64, V=64)
    s.update(kw)
    return [s[n] for n in "BLHGKV"]


def test_ckpt_size(lib):
    from mamba_selective_ssm_gb300 import _capi as c
    mp32, mp16 = 2 * 64 * 64 + 272, 3 * 64 * 64 + 272  # a chunk's two 64 x 64 operands and scalars
    assert lib.deltarule_ckpt_size(64, 32, 40, c.SS_F32) == 2 * 32 * 40 + 2 * 64 * 40 + mp32  # two states, r and o
    assert lib.deltarule_ckpt_size(65, 32, 40, c.SS_F32) == 3 * 32 * 40 + 2 * 128 * 40 + 2 * mp32
    assert lib.deltarule_ckpt_size(65, 32, 40, c.SS_BF16) == 3 * 32 * 40 + 2 * 128 * 40 + 2 * mp16
    for bad in ((0, 32, 40, 0), (64, 30, 40, 0), (64, 32, 136, 0), (64, 32, 40, 2)):
        assert lib.deltarule_ckpt_size(*bad) == 0


@pytest.mark.parametrize("dt", [0, 1])
def test_fwd_refusals(lib, dt):
    from mamba_selective_ssm_gb300 import _capi as c

    def call(ptr=None, at=None, ld=(128, 128, 256), dt=dt, ws=WS, wsz=1 << 40, **kw):
        q = list(P[:10])  # q k v g beta h0 lengths o ckpt h_last
        if at is not None:
            q[at] = ptr
        return lib.deltarule_fwd(q[0], ld[0], q[1], ld[1], q[2], ld[2], *q[3:], *_sizes(**kw), 0.1, dt, ws, wsz, None)

    for at in (0, 1, 2, 4, 7):
        assert call(None, at) == c.SS_ERR_NULL
    for n in "BLHGKV":
        assert call(**{n: 0}) == c.SS_ERR_DIM
        assert call(**{n: -1}) == c.SS_ERR_DIM
    assert call(H=5) == c.SS_ERR_DIM
    assert call(K=60) == c.SS_ERR_ALIGN
    assert call(V=12) == c.SS_ERR_ALIGN
    assert call(K=136) == c.SS_ERR_DIM
    assert call(V=136) == c.SS_ERR_DIM
    assert call(L=INT_MAX) == c.SS_ERR_DIM
    assert call(B=1 << 20, H=32, G=2, L=1, ld=(128, 128, 2048)) == c.SS_ERR_DIM
    assert call(B=1 << 16, L=1 << 16) == c.SS_ERR_DIM
    assert call(dt=7) == c.SS_ERR_UNSUPPORTED
    assert call(ld=(120, 128, 256)) == c.SS_ERR_DIM
    assert call(ld=(128, 132, 256)) == c.SS_ERR_ALIGN
    assert call(ld=(128, 128, 255)) == c.SS_ERR_DIM
    for at in (0, 1, 2, 5, 7, 8, 9):
        assert call(_fake(0x100008), at) == c.SS_ERR_ALIGN
    for at in (3, 4, 6):
        assert call(_fake(0x100002), at) == c.SS_ERR_ALIGN
    need = lib.deltarule_fwd_workspace_size(*_sizes(), dt)
    assert need > 0 and lib.deltarule_fwd_workspace_size(*_sizes(K=4), dt) == 0
    assert call(None, 8, ws=None) == c.SS_ERR_WORKSPACE  # (with ckpt there is no workspace)
    assert call(None, 8, wsz=need - 1) == c.SS_ERR_WORKSPACE
    assert call(None, 8, ws=_fake(0x900008)) == c.SS_ERR_ALIGN


@pytest.mark.parametrize("dt", [0, 1])
def test_bwd_refusals(lib, dt):
    from mamba_selective_ssm_gb300 import _capi as c

    def call(ptr=None, at=None, ld=(128, 128, 256), dt=dt, ws=WS, wsz=1 << 40, **kw):
        q = list(P[:15])  # q k v g beta lengths ckpt dout dh_last dq dk dv dg dbeta dh0
        if at is not None:
            q[at] = ptr
        return lib.deltarule_bwd(q[0], ld[0], q[1], ld[1], q[2], ld[2], *q[3:], *_sizes(**kw), 0.1, dt, ws, wsz, None)

    for at in (0, 1, 2, 4, 6, 7, 9, 10, 11, 12, 13):
        assert call(None, at) == c.SS_ERR_NULL
    assert call(H=3) == c.SS_ERR_DIM
    assert call(K=12) == c.SS_ERR_ALIGN
    assert call(V=256) == c.SS_ERR_DIM
    assert call(dt=2) == c.SS_ERR_UNSUPPORTED
    assert call(ld=(128, 128, 248)) == c.SS_ERR_DIM
    for at in (0, 6, 7, 8, 9, 10, 11, 14):
        assert call(_fake(0x100008), at) == c.SS_ERR_ALIGN
    for at in (3, 4, 5, 12, 13):
        assert call(_fake(0x100002), at) == c.SS_ERR_ALIGN
    need = lib.deltarule_bwd_workspace_size(*_sizes(), dt)
    assert need >= 2 * 2 * 100 * 4 * 64 * 4  # heads share q, k: one fp32 part of dq and dk for each head
    assert call(ws=None) == c.SS_ERR_WORKSPACE
    assert call(wsz=need - 1) == c.SS_ERR_WORKSPACE
    assert lib.deltarule_bwd_workspace_size(*_sizes(B=0), dt) == 0


def test_step_refusals(lib):
    from mamba_selective_ssm_gb300 import _capi as c
    call = lambda p=P, B=2, H=4, G=2, K=64, V=64, dt=c.SS_BF16: lib.deltarule_step(*p[:7], B, H, G, K, V, 0.1, dt, None)
    for at in (0, 1, 2, 4, 5, 6):
        q = list(P)
        q[at] = None
        assert call(q) == c.SS_ERR_NULL
    assert call(B=0) == c.SS_ERR_DIM
    assert call(G=3) == c.SS_ERR_DIM
    assert call(K=9) == c.SS_ERR_ALIGN
    assert call(V=1024) == c.SS_ERR_DIM
    assert call(B=INT_MAX, H=4) == c.SS_ERR_DIM
    assert call(dt=3) == c.SS_ERR_UNSUPPORTED
    for at, addr in ((5, 0x100004), (0, 0x100008), (3, 0x100002), (4, 0x100001)):
        q = list(P)
        q[at] = _fake(addr)
        assert call(q) == c.SS_ERR_ALIGN


def test_groupnorm_refusals(lib):
    from mamba_selective_ssm_gb300 import _capi as c

    def fwd(p=P, N=2, M=100, C=64, groups=8, eps=1e-5, dt=c.SS_BF16, ws=WS, wsz=1 << 40):
        return lib.groupnorm_fwd(*p[:3], eps, *p[3:6], N, M, C, groups, 1, dt, ws, wsz, None)

    def bwd(p=P, N=2, M=100, C=64, groups=8, dt=c.SS_BF16, ws=WS, wsz=1 << 40):
        return lib.groupnorm_bwd(*p[:9], 0, N, M, C, groups, 1, dt, ws, wsz, None)

    for call, need in ((fwd, (0, 1, 3)), (bwd, (0, 1, 2, 4, 5, 6, 7, 8))):
        for at in need:
            q = list(P)
            q[at] = None
            assert call(q) == c.SS_ERR_NULL
        for kw in (dict(N=0), dict(M=0), dict(C=0), dict(groups=0), dict(N=-1), dict(C=32776), dict(groups=7), dict(groups=65), dict(N=INT_MAX),
                   dict(M=INT_MAX), dict(N=1 << 28, groups=8), dict(N=1 << 20, M=1 << 20)):
            assert call(**kw) == c.SS_ERR_DIM, kw
        assert call(C=60, groups=4) == c.SS_ERR_ALIGN
        assert call(dt=4) == c.SS_ERR_UNSUPPORTED
    assert fwd(eps=-1.0) == c.SS_ERR_DIM
    assert fwd(eps=float("nan")) == c.SS_ERR_DIM
    for call, ats in ((fwd, (0, 1, 2, 3)), (bwd, (0, 1, 2, 3, 6))):
        for at in ats:
            q = list(P)
            q[at] = _fake(0x100008)
            assert call(q) == c.SS_ERR_ALIGN
    for call, ats in ((fwd, (4, 5)), (bwd, (4, 5, 7, 8))):
        for at in ats:
            q = list(P)
            q[at] = _fake(0x100002)
            assert call(q) == c.SS_ERR_ALIGN
    # long samples are summed in parts, which need scratch; a token's groups are not
    need = lib.groupnorm_fwd_workspace_size(2, 5000, 512, 8, c.SS_BF16)
    assert need > 0 and lib.groupnorm_fwd_workspace_size(100, 1, 512, 8, c.SS_BF16) == 0
    big = dict(N=2, M=5000, C=512, groups=8)
    assert fwd(**big, ws=None) == c.SS_ERR_WORKSPACE and fwd(**big, wsz=need - 1) == c.SS_ERR_WORKSPACE
    assert fwd(**big, ws=_fake(0x900008)) == c.SS_ERR_ALIGN
    need = lib.groupnorm_bwd_workspace_size(2, 100, 64, 8, c.SS_BF16)
    assert need > 0 and lib.groupnorm_bwd_workspace_size(2, 100, 64, 7, c.SS_BF16) == 0
    assert bwd(ws=None) == c.SS_ERR_WORKSPACE and bwd(wsz=need - 1) == c.SS_ERR_WORKSPACE
    assert bwd(ws=_fake(0x900008)) == c.SS_ERR_ALIGN
