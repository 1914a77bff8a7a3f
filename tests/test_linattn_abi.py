"""Refusals of the linear attention and layer norm entry points: the documented status before anything is launched
(CPU), and the Python layer's checks."""

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


def _sizes(**kw):
    s = dict(B=2, L=100, H=4, G=2, K=64, V=64)
    s.update(kw)
    return [s[n] for n in "BLHGKV"]


def test_num_chunks(lib):
    from mamba_selective_ssm_gb300 import _capi as c
    for dt in (c.SS_F32, c.SS_BF16):
        n = lib.linattn_num_chunks(1, dt)
        assert n == 1 and lib.linattn_num_chunks(0, dt) == 0 and lib.linattn_num_chunks(4096, dt) >= 32
    assert lib.linattn_num_chunks(10, 5) == 0


def test_fwd_refusals(lib):
    from mamba_selective_ssm_gb300 import _capi as c

    def call(ptr=None, at=None, ld=(128, 128, 256), dt=c.SS_BF16, ws=WS, wsz=1 << 40, **kw):
        q = list(P[:9])  # q k v g h0 lengths o ckpt h_last
        if at is not None:
            q[at] = ptr
        return lib.linattn_fwd(q[0], ld[0], q[1], ld[1], q[2], ld[2], q[3], 0, q[4], q[5], q[6], q[7], q[8], *_sizes(**kw), 0.1, dt,
                               ws, wsz, None)

    for at in (0, 1, 2, 3, 6):
        assert call(None, at) == c.SS_ERR_NULL
    for n in "BLHGKV":
        assert call(**{n: 0}) == c.SS_ERR_DIM
    assert call(H=5) == c.SS_ERR_DIM
    assert call(K=60) == c.SS_ERR_ALIGN
    assert call(V=12) == c.SS_ERR_ALIGN
    assert call(K=136) == c.SS_ERR_DIM
    assert call(V=136) == c.SS_ERR_DIM
    assert call(dt=7) == c.SS_ERR_UNSUPPORTED
    assert call(ld=(120, 128, 256)) == c.SS_ERR_DIM
    assert call(ld=(128, 132, 256)) == c.SS_ERR_ALIGN
    assert call(ld=(128, 128, 255)) == c.SS_ERR_DIM
    assert call(_fake(0x100008), 0) == c.SS_ERR_ALIGN
    assert call(_fake(0x100008), 7) == c.SS_ERR_ALIGN
    assert call(_fake(0x100002), 3) == c.SS_ERR_ALIGN
    assert call(_fake(0x100002), 5) == c.SS_ERR_ALIGN
    # one long row is cut in segments, which need scratch; many rows are not
    need = lib.linattn_fwd_workspace_size(*_sizes(B=1, L=16384), c.SS_BF16)
    assert need > 0
    assert lib.linattn_fwd_workspace_size(*_sizes(B=256, L=512), c.SS_BF16) == 0
    assert lib.linattn_fwd_workspace_size(*_sizes(K=4), c.SS_BF16) == 0
    assert call(B=1, L=16384, ws=None) == c.SS_ERR_WORKSPACE
    assert call(B=1, L=16384, wsz=need - 1) == c.SS_ERR_WORKSPACE
    assert call(B=1, L=16384, ws=_fake(0x900008)) == c.SS_ERR_ALIGN


def test_bwd_refusals(lib):
    from mamba_selective_ssm_gb300 import _capi as c

    def call(ptr=None, at=None, ld=(128, 128, 256), dt=c.SS_F32, ws=WS, wsz=1 << 40, **kw):
        q = list(P[:13])  # q k v g lengths ckpt dout dh_last dq dk dv dg dh0
        if at is not None:
            q[at] = ptr
        return lib.linattn_bwd(q[0], ld[0], q[1], ld[1], q[2], ld[2], q[3], 0, *q[4:], *_sizes(**kw), 0.1, dt, ws, wsz, None)

    for at in (0, 1, 2, 3, 5, 6, 8, 9, 10, 11):
        assert call(None, at) == c.SS_ERR_NULL
    assert call(H=3) == c.SS_ERR_DIM
    assert call(K=12) == c.SS_ERR_ALIGN
    assert call(V=256) == c.SS_ERR_DIM
    assert call(dt=2) == c.SS_ERR_UNSUPPORTED
    assert call(ld=(128, 128, 248)) == c.SS_ERR_DIM
    assert call(_fake(0x100008), 9) == c.SS_ERR_ALIGN
    need = lib.linattn_bwd_workspace_size(*_sizes(), 0, c.SS_F32)
    assert need >= 2 * 2 * 100 * 4 * 64 * 4  # heads share q, k: one fp32 part of dq and dk for each head
    assert call(ws=None) == c.SS_ERR_WORKSPACE
    assert call(wsz=need - 1) == c.SS_ERR_WORKSPACE
    assert lib.linattn_bwd_workspace_size(*_sizes(), 1, c.SS_F32) > need  # per-chunk sums of dg
    assert lib.linattn_bwd_workspace_size(*_sizes(B=0), 0, c.SS_F32) == 0


def test_step_refusals(lib):
    from mamba_selective_ssm_gb300 import _capi as c
    call = lambda p=P, B=2, H=4, G=2, K=64, V=64, dt=c.SS_BF16: lib.linattn_step(*p[:4], 0, *p[4:6], B, H, G, K, V, 0.1, dt, None)
    for at in range(6):
        q = list(P)
        q[at] = None
        assert call(q) == c.SS_ERR_NULL
    assert call(B=0) == c.SS_ERR_DIM
    assert call(G=3) == c.SS_ERR_DIM
    assert call(K=9) == c.SS_ERR_ALIGN
    assert call(V=1024) == c.SS_ERR_DIM
    assert call(dt=3) == c.SS_ERR_UNSUPPORTED
    q = list(P)
    q[4] = _fake(0x100004)
    assert call(q) == c.SS_ERR_ALIGN


def test_layernorm_refusals(lib):
    from mamba_selective_ssm_gb300 import _capi as c
    fwd = lambda p=P, eps=1e-5, R=4, N=64, dt=c.SS_F32: lib.layernorm_fwd(*p[:3], eps, *p[3:6], R, N, dt, None)
    for at in (0, 1, 3):
        q = list(P)
        q[at] = None
        assert fwd(q) == c.SS_ERR_NULL
    assert fwd(eps=-1.0) == c.SS_ERR_DIM
    assert fwd(eps=float("nan")) == c.SS_ERR_DIM
    assert fwd(R=0) == c.SS_ERR_DIM
    assert fwd(N=12) == c.SS_ERR_ALIGN
    assert fwd(N=32776) == c.SS_ERR_DIM
    assert fwd(dt=2) == c.SS_ERR_UNSUPPORTED
    q = list(P)
    q[2] = _fake(0x100008)
    assert fwd(q) == c.SS_ERR_ALIGN
    need = lib.layernorm_bwd_workspace_size(100, 768)
    assert need > 0 and lib.layernorm_bwd_workspace_size(100, 770) == 0
    bwd = lambda p=P, R=100, N=768, dt=c.SS_BF16, ws=WS, wsz=need: lib.layernorm_bwd(*p[:8], 0, R, N, dt, ws, wsz, None)
    for at in range(8):
        q = list(P)
        q[at] = None
        assert bwd(q) == c.SS_ERR_NULL
    assert bwd(ws=None) == c.SS_ERR_WORKSPACE
    assert bwd(wsz=need - 4) == c.SS_ERR_WORKSPACE
    assert bwd(ws=_fake(0x900004)) == c.SS_ERR_ALIGN
    assert bwd(N=4) == c.SS_ERR_ALIGN


def test_wrappers_refuse_cpu_tensors(lib):
    torch = pytest.importorskip("torch")
    import mamba_selective_ssm_gb300 as ss
    q, v, g = torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2, 8), torch.zeros(1, 4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ss.linattn_fwd(q, q, v, g)
    with pytest.raises(ValueError, match="CUDA"):
        ss.linattn_step(q[:, 0], q[:, 0], v[:, 0], g[:, 0], torch.zeros(1, 2, 8, 8))
    with pytest.raises(ValueError, match="CUDA"):
        ss.layernorm_fwd(torch.zeros(2, 8), torch.ones(8), None, 1e-5)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ss.linattn_fwd(q.half(), q.half(), v.half(), g)
    with pytest.raises(ValueError, match=r"\[B, L, G, K\]"):
        ss.linattn_fwd(q[0], q[0], v, g)
