"""PyTorch-facing calls of libssscan: argument checks, output allocation and the
C-ABI call on the current CUDA stream.  No arithmetic of the method is done here.

Names and argument order follow include/ssscan.h:

* ``ss_scan_fwd(x, delta, A, Bm, Cm, Dv, z, h0=None, chunk=64, workspace=None)``
  -> ``(y, ckpt, h_last)``
* ``ss_scan_bwd(x, delta, A, Bm, Cm, Dv, z, ckpt, dy, dh_last=None, chunk=64, dA=None, dD=None, ...)``
  -> dict of gradients
* ``conv1d_causal_bwd(dout, x, w, dw=None, db=None)`` -> ``(dx, dw, db)``
* ``rmsnorm_bwd(dy, x, scale, rms, dscale=None)`` -> ``(dx, dscale)``
* ``conv1d_causal_fwd(x, w, bias=None, silu=False)`` -> ``out``
* ``conv1d_causal_silu_bwd(dact, x, w, bias=None, dw=None, db=None)`` -> ``(dx, dw, db)``
* ``rmsnorm_fwd(x, scale, eps)`` -> ``(y, rms)``
* ``ss_scan_step(x, delta, A, Bm, Cm, Dv, z, h)`` -> ``y`` (h updated in place)
* ``ss_scan_fwd_summary(x, delta, A, Bm)`` -> ``(h_end, delta_sum)``;
  ``ss_scan_bwd_summary(delta, A, Cm, z, dy)`` -> ``(g_start, delta_sum)``;
  ``ss_scan_carries(A, delta_sum, summ, init=None, reverse=False)`` -> ``carry``
  (the pieces of a sequence-sharded scan; ``sharded.py`` runs them over ranks)
* ``conv1d_causal_step(x, conv_state, w, bias=None, silu=False)`` -> ``out`` (state updated in place)
* ``linattn_fwd(q, k, v, g, h0=None, scale=None, lengths=None)`` -> ``(o, ckpt, h_last)``
* ``linattn_bwd(q, k, v, g, ckpt, do, dh_last=None, scale=None, lengths=None)`` -> dict of gradients
* ``linattn_step(q, k, v, g, h, scale=None)`` -> ``o`` (h updated in place)
* ``layernorm_fwd(x, scale, bias, eps)`` -> ``(y, mean, rstd)``
* ``layernorm_bwd(dy, x, scale, mean, rstd, dscale=None, dbias=None)`` -> ``(dx, dscale, dbias)``

Activations are ``torch.float32`` or ``torch.bfloat16`` CUDA tensors, contiguous;
parameters, states and gradients are ``torch.float32``.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _capi
from ._capi import SS_BF16, SS_F32, check, load

_DT = {torch.float32: SS_F32, torch.bfloat16: SS_BF16}


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _req(t, name, shape=None, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (strided views are not accepted)")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _act_dtype(x):
    if x.dtype not in _DT:
        raise ValueError(f"activations must be float32 or bfloat16, got {x.dtype}")
    return _DT[x.dtype]


def num_chunks(L: int, chunk: int) -> int:
    return load().ss_scan_num_chunks(L, chunk)


def scan_fwd_workspace_size(B, L, D, N, chunk, dtype) -> int:
    return load().ss_scan_fwd_workspace_size(B, L, D, N, chunk, _DT[dtype])


def ss_scan_fwd(x, delta, A, Bm, Cm, Dv, z, h0=None, chunk: int = 64, want_h_last: bool = True, workspace=None,
                dt_bias=None, delta_softplus: bool = False):
    """Forward scan -> ``(y, ckpt, h_last)``.  With ``dt_bias`` / ``delta_softplus`` the
    recurrence uses softplus(delta + dt_bias) (or delta + dt_bias), computed in the kernel."""
    lib = load()
    B, L, D = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    _act_dtype(x)
    for name, t in (("x", x), ("delta", delta), ("z", z)):
        _req(t, name, (B, L, D), dt, dev)
    for name, t in (("Bm", Bm), ("Cm", Cm)):
        _req(t, name, (B, L, N), dt, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    _req(Dv, "Dv", (D,), torch.float32, dev)
    if h0 is not None:
        _req(h0, "h0", (B, D, N), torch.float32, dev)
    if dt_bias is not None:
        _req(dt_bias, "dt_bias", (D,), torch.float32, dev)
    nck = num_chunks(L, chunk) if L > 0 and chunk > 0 else 0
    y = torch.empty_like(x)
    ckpt = torch.empty((B, max(nck, 1), D, N), device=dev, dtype=torch.float32)
    h_last = torch.empty((B, D, N), device=dev, dtype=torch.float32) if want_h_last else None
    ws_bytes = lib.ss_scan_fwd_workspace_size(B, L, D, N, chunk, _DT[dt])
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, device=dev, dtype=torch.uint8)
    ws_have = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib.ss_scan_fwd(_p(x), _p(delta), _p(A), _p(Bm), _p(Cm), _p(Dv), _p(z), _p(h0), _p(y), _p(ckpt), _p(h_last),
                         B, L, D, N, chunk, _DT[dt], _p(dt_bias), int(bool(delta_softplus)), _p(workspace), ws_have,
                         _stream())
    check(rc, "ss_scan_fwd")
    return y, ckpt, h_last


def scan_bwd_workspace_size(B, L, D, N, chunk, dtype) -> int:
    return load().ss_scan_bwd_workspace_size(B, L, D, N, chunk, _DT[dtype])


def ss_scan_bwd(x, delta, A, Bm, Cm, Dv, z, ckpt, dy, dh_last=None, chunk: int = 64, dA=None, dD=None,
                want_dh0: bool = True, workspace=None, out=None, dt_bias=None, delta_softplus: bool = False,
                d_dt_bias=None):
    """Gradients of sum(y*dy) (+ sum(h_last*dh_last)).  dA and dD accumulate into the
    given tensors (zeros when None); the rest are returned freshly (or written into ``out``).
    With the fused discretisation (same ``dt_bias`` / ``delta_softplus`` as the forward),
    ``ddelta`` is the gradient of the raw delta and ``d_dt_bias`` accumulates (zeros when None)."""
    lib = load()
    B, L, D = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    _act_dtype(x)
    for name, t in (("x", x), ("delta", delta), ("z", z), ("dy", dy)):
        _req(t, name, (B, L, D), dt, dev)
    for name, t in (("Bm", Bm), ("Cm", Cm)):
        _req(t, name, (B, L, N), dt, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    _req(Dv, "Dv", (D,), torch.float32, dev)
    _req(ckpt, "ckpt", (B, num_chunks(L, chunk), D, N), torch.float32, dev)
    if dh_last is not None:
        _req(dh_last, "dh_last", (B, D, N), torch.float32, dev)
    f32 = dict(device=dev, dtype=torch.float32)
    if out is None:
        out = {
            "dx": torch.empty((B, L, D), **f32), "ddelta": torch.empty((B, L, D), **f32),
            "dz": torch.empty((B, L, D), **f32), "dB": torch.empty((B, L, N), **f32),
            "dC": torch.empty((B, L, N), **f32),
            "dh0": torch.empty((B, D, N), **f32) if want_dh0 else None,
        }
    fused = dt_bias is not None or delta_softplus
    if dt_bias is not None:
        _req(dt_bias, "dt_bias", (D,), torch.float32, dev)
    if fused:
        out["d_dt_bias"] = (torch.zeros((D,), **f32) if d_dt_bias is None
                            else _req(d_dt_bias, "d_dt_bias", (D,), torch.float32, dev))
    out["dA"] = torch.zeros((D, N), **f32) if dA is None else _req(dA, "dA", (D, N), torch.float32, dev)
    out["dD"] = torch.zeros((D,), **f32) if dD is None else _req(dD, "dD", (D,), torch.float32, dev)
    ws_bytes = lib.ss_scan_bwd_workspace_size(B, L, D, N, chunk, _DT[dt])
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=dev, dtype=torch.uint8)
    rc = lib.ss_scan_bwd(_p(x), _p(delta), _p(A), _p(Bm), _p(Cm), _p(Dv), _p(z), _p(ckpt), _p(dy), _p(dh_last),
                         _p(out["dx"]), _p(out["ddelta"]), _p(out["dz"]), _p(out["dA"]), _p(out["dB"]), _p(out["dC"]),
                         _p(out["dD"]), _p(out.get("dh0")), B, L, D, N, chunk, _DT[dt], _p(dt_bias),
                         int(bool(delta_softplus)), _p(out.get("d_dt_bias")), _p(workspace),
                         workspace.numel() * workspace.element_size(), _stream())
    check(rc, "ss_scan_bwd")
    return out


def ss_scan_fwd_summary(x, delta, A, Bm, dt_bias=None, delta_softplus: bool = False):
    """Forward summary of one piece of a sequence -> ``(h_end [B,D,N], delta_sum [B,D])``:
    the state the piece reaches from a zero start and its sum of (discretised) delta."""
    lib = load()
    B, L, D = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    _act_dtype(x)
    _req(x, "x", (B, L, D), dt, dev)
    _req(delta, "delta", (B, L, D), dt, dev)
    _req(Bm, "Bm", (B, L, N), dt, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    if dt_bias is not None:
        _req(dt_bias, "dt_bias", (D,), torch.float32, dev)
    h_end = torch.empty((B, D, N), device=dev, dtype=torch.float32)
    dsum = torch.empty((B, D), device=dev, dtype=torch.float32)
    rc = lib.ss_scan_fwd_summary(_p(x), _p(delta), _p(A), _p(Bm), _p(h_end), _p(dsum), B, L, D, N, _DT[dt],
                                 _p(dt_bias), int(bool(delta_softplus)), _stream())
    check(rc, "ss_scan_fwd_summary")
    return h_end, dsum


def ss_scan_bwd_summary(delta, A, Cm, z, dy, dt_bias=None, delta_softplus: bool = False):
    """Backward summary of one piece -> ``(g_start [B,D,N], delta_sum [B,D])``: the adjoint the
    piece sends out of its first step when no carry arrives at its end, and its sum of delta."""
    lib = load()
    B, L, D = delta.shape
    N = A.shape[1]
    dev, dt = delta.device, delta.dtype
    _act_dtype(delta)
    for name, t in (("delta", delta), ("z", z), ("dy", dy)):
        _req(t, name, (B, L, D), dt, dev)
    _req(Cm, "Cm", (B, L, N), dt, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    if dt_bias is not None:
        _req(dt_bias, "dt_bias", (D,), torch.float32, dev)
    g_start = torch.empty((B, D, N), device=dev, dtype=torch.float32)
    dsum = torch.empty((B, D), device=dev, dtype=torch.float32)
    rc = lib.ss_scan_bwd_summary(_p(delta), _p(A), _p(Cm), _p(z), _p(dy), _p(g_start), _p(dsum), B, L, D, N, _DT[dt],
                                 _p(dt_bias), int(bool(delta_softplus)), _stream())
    check(rc, "ss_scan_bwd_summary")
    return g_start, dsum


def ss_scan_carries(A, delta_sum, summ, init=None, reverse: bool = False):
    """Compose P pieces' affine maps (piece-major ``delta_sum [P,B,D]``, ``summ [P,B,D,N]``)
    -> ``carry [P,B,D,N]``: the state entering each piece (forward) or the carry arriving
    at its end (``reverse``), starting from ``init`` (zeros when None)."""
    lib = load()
    P, B, D, N = summ.shape
    dev = summ.device
    _req(A, "A", (D, N), torch.float32, dev)
    _req(delta_sum, "delta_sum", (P, B, D), torch.float32, dev)
    _req(summ, "summ", (P, B, D, N), torch.float32, dev)
    if init is not None:
        _req(init, "init", (B, D, N), torch.float32, dev)
    carry = torch.empty((P, B, D, N), device=dev, dtype=torch.float32)
    rc = lib.ss_scan_carries(_p(A), _p(delta_sum), _p(summ), _p(init), _p(carry), P, B, D, N, int(bool(reverse)),
                             _stream())
    check(rc, "ss_scan_carries")
    return carry


def conv1d_causal_bwd(dout, x, w, dw=None, db=None, workspace=None):
    lib = load()
    B, L, D = x.shape
    K = w.shape[1]
    dev = x.device
    xdt = _act_dtype(x)
    _req(dout, "dout", (B, L, D), torch.float32, dev)
    _req(x, "x", (B, L, D), x.dtype, dev)
    _req(w, "w", (D, K), torch.float32, dev)
    dw = torch.zeros((D, K), device=dev, dtype=torch.float32) if dw is None else _req(dw, "dw", (D, K), torch.float32, dev)
    db = torch.zeros((D,), device=dev, dtype=torch.float32) if db is None else _req(db, "db", (D,), torch.float32, dev)
    dx = torch.empty((B, L, D), device=dev, dtype=torch.float32)
    ws_bytes = lib.conv1d_causal_bwd_workspace_size(B, L, D, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=dev, dtype=torch.uint8)
    rc = lib.conv1d_causal_bwd(_p(dout), _p(x), _p(w), _p(dx), _p(dw), _p(db), B, L, D, K, xdt, _p(workspace),
                               workspace.numel() * workspace.element_size(), _stream())
    check(rc, "conv1d_causal_bwd")
    return dx, dw, db


def conv1d_causal_silu_bwd(dact, x, w, bias=None, dw=None, db=None, workspace=None):
    """Backward through silu(conv1d(x) + bias) given dL/d(silu output); dw, db accumulate."""
    lib = load()
    B, L, D = x.shape
    K = w.shape[1]
    dev = x.device
    xdt = _act_dtype(x)
    _req(dact, "dact", (B, L, D), torch.float32, dev)
    _req(x, "x", (B, L, D), x.dtype, dev)
    _req(w, "w", (D, K), torch.float32, dev)
    if bias is not None:
        _req(bias, "bias", (D,), torch.float32, dev)
    dw = torch.zeros((D, K), device=dev, dtype=torch.float32) if dw is None else _req(dw, "dw", (D, K), torch.float32, dev)
    db = torch.zeros((D,), device=dev, dtype=torch.float32) if db is None else _req(db, "db", (D,), torch.float32, dev)
    dx = torch.empty((B, L, D), device=dev, dtype=torch.float32)
    ws_bytes = lib.conv1d_causal_bwd_workspace_size(B, L, D, K)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=dev, dtype=torch.uint8)
    rc = lib.conv1d_causal_silu_bwd(_p(dact), _p(x), _p(w), _p(bias), _p(dx), _p(dw), _p(db), B, L, D, K, xdt,
                                    _p(workspace), workspace.numel() * workspace.element_size(), _stream())
    check(rc, "conv1d_causal_silu_bwd")
    return dx, dw, db


def rmsnorm_bwd(dy, x, scale, rms, dscale=None, workspace=None):
    lib = load()
    R, H = x.shape
    dev = x.device
    dt = _act_dtype(x)
    _req(dy, "dy", (R, H), x.dtype, dev)
    _req(x, "x", (R, H), x.dtype, dev)
    _req(scale, "scale", (H,), torch.float32, dev)
    _req(rms, "rms", (R,), torch.float32, dev)
    dscale = torch.zeros((H,), device=dev, dtype=torch.float32) if dscale is None else _req(
        dscale, "dscale", (H,), torch.float32, dev)
    dx = torch.empty((R, H), device=dev, dtype=torch.float32)
    ws_bytes = lib.rmsnorm_bwd_workspace_size(R, H)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 16), device=dev, dtype=torch.uint8)
    rc = lib.rmsnorm_bwd(_p(dy), _p(x), _p(scale), _p(rms), _p(dx), _p(dscale), R, H, dt, _p(workspace),
                         workspace.numel() * workspace.element_size(), _stream())
    check(rc, "rmsnorm_bwd")
    return dx, dscale


def conv1d_causal_fwd(x, w, bias=None, silu: bool = False, out=None):
    """Depthwise causal conv1d (+ optional SiLU); ``out`` has x's dtype."""
    lib = load()
    B, L, D = x.shape
    K = w.shape[1]
    dev = x.device
    xdt = _act_dtype(x)
    _req(x, "x", (B, L, D), x.dtype, dev)
    _req(w, "w", (D, K), torch.float32, dev)
    if bias is not None:
        _req(bias, "bias", (D,), torch.float32, dev)
    out = torch.empty_like(x) if out is None else _req(out, "out", (B, L, D), x.dtype, dev)
    rc = lib.conv1d_causal_fwd(_p(x), _p(w), _p(bias), _p(out), B, L, D, K, int(bool(silu)), xdt, _stream())
    check(rc, "conv1d_causal_fwd")
    return out


def rmsnorm_fwd(x, scale, eps: float, want_rms: bool = True):
    """RMSNorm forward: ``(y, rms)`` with y in x's dtype and rms fp32 (None unless ``want_rms``)."""
    lib = load()
    R, H = x.shape
    dev = x.device
    dt = _act_dtype(x)
    _req(x, "x", (R, H), x.dtype, dev)
    _req(scale, "scale", (H,), torch.float32, dev)
    y = torch.empty_like(x)
    rms = torch.empty((R,), device=dev, dtype=torch.float32) if want_rms else None
    rc = lib.rmsnorm_fwd(_p(x), _p(scale), float(eps), _p(y), _p(rms), R, H, dt, _stream())
    check(rc, "rmsnorm_fwd")
    return y, rms


def ss_scan_step(x, delta, A, Bm, Cm, Dv, z, h):
    """One decode step for B sequences: updates ``h`` [B,D,N] in place and returns y [B,D]."""
    lib = load()
    B, D = x.shape
    N = A.shape[1]
    dev, dt = x.device, x.dtype
    _act_dtype(x)
    for name, t in (("x", x), ("delta", delta), ("z", z)):
        _req(t, name, (B, D), dt, dev)
    for name, t in (("Bm", Bm), ("Cm", Cm)):
        _req(t, name, (B, N), dt, dev)
    _req(A, "A", (D, N), torch.float32, dev)
    _req(Dv, "Dv", (D,), torch.float32, dev)
    _req(h, "h", (B, D, N), torch.float32, dev)
    y = torch.empty_like(x)
    rc = lib.ss_scan_step(_p(x), _p(delta), _p(A), _p(Bm), _p(Cm), _p(Dv), _p(z), _p(h), _p(y), B, D, N, _DT[dt],
                          _stream())
    check(rc, "ss_scan_step")
    return y


def conv1d_causal_step(x, conv_state, w, bias=None, silu: bool = False):
    """One conv step for B sequences: shifts ``conv_state`` [B,D,K] in place and returns out [B,D]."""
    lib = load()
    B, D = x.shape
    K = w.shape[1]
    dev = x.device
    xdt = _act_dtype(x)
    _req(conv_state, "conv_state", (B, D, K), torch.float32, dev)
    _req(w, "w", (D, K), torch.float32, dev)
    if bias is not None:
        _req(bias, "bias", (D,), torch.float32, dev)
    out = torch.empty_like(x)
    rc = lib.conv1d_causal_step(_p(x), _p(conv_state), _p(w), _p(bias), _p(out), B, D, K, int(bool(silu)), xdt,
                                _stream())
    check(rc, "conv1d_causal_step")
    return out


def linattn_num_chunks(L: int, dtype) -> int:
    """Checkpoints a row of L tokens has (``ckpt`` is [B, H, that, K, V])."""
    return load().linattn_num_chunks(L, _DT[dtype])


# The calls below take a few microseconds on the GPU at their smallest, so their Python is kept short: a tensor
# that is as expected passes one test, sizes of scratch are kept by the sizes they follow from, and pointers and the
# stream go to ctypes as integers.


def _raw_stream(dev):
    """The current stream's handle.  The library launches on the current device, so that is where the tensors must be: on
    another one their addresses and their stream would belong to a device that runs nothing here."""
    current = torch.cuda.current_device()
    if dev.index != current:
        raise ValueError(f"the tensors are on {dev}, but the current device is cuda:{current}")
    return torch._C._cuda_getCurrentRawStream(current)


def _at(t, name, shape, dtype, dev):
    """The address of a dense tensor of this shape, type and device (``_req``'s errors for any other)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.get_device() == dev.index
            and t.is_contiguous()):
        _req(t, name, shape, dtype, dev)
    return t.data_ptr()


def _opt_at(t, name, shape, dtype, dev):
    return None if t is None else _at(t, name, shape, dtype, dev)


def _rows(t, name, shape, dtype, dev):
    """A [B, L, heads, width] input whose tokens may lie further apart than their own rows (a column range of a
    wider [B, L, W] array): its address and its token stride in elements."""
    B, L, n, w = shape
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda and t.get_device() == dev.index:
        if t.is_contiguous():
            return t.data_ptr(), n * w
    elif not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    elif not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    elif t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    elif t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    else:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    sb, sl, sn, sw = t.stride()
    if L == 1:
        sl = sb if B > 1 else n * w  # one token a row: rows are the batch's
    if (w > 1 and sw != 1) or (n > 1 and sn != w) or (B > 1 and L > 0 and sb != L * sl):
        raise ValueError(f"{name} must hold each token's heads contiguously and its batch rows L tokens apart, got "
                         f"strides {t.stride()}")
    return t.data_ptr(), sl


@functools.lru_cache(maxsize=1024)
def _linattn_plan(B, L, H, G, K, V, per_head, sdt):
    """(chunks, forward scratch, backward scratch) of a call's sizes."""
    lib = load()
    return (lib.linattn_num_chunks(L, sdt), lib.linattn_fwd_workspace_size(B, L, H, G, K, V, sdt),
            lib.linattn_bwd_workspace_size(B, L, H, G, K, V, per_head, sdt))


@functools.lru_cache(maxsize=1024)
def _layernorm_plan(R, N):
    return load().layernorm_bwd_workspace_size(R, N)


def _linattn_sizes(q, v):
    if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor):
        raise TypeError("q, k, v must be torch.Tensor")
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"q, k must be [B, L, G, K] and v [B, L, H, V], got {tuple(q.shape)} and {tuple(v.shape)}")
    B, L, G, K = q.shape
    return B, L, v.shape[2], G, K, v.shape[3]


def _linattn_gate(g, B, L, H, dev):
    """The address of g, and 1 when it has one log decay for each head, 0 when one for each token."""
    if isinstance(g, torch.Tensor) and g.dim() == 1:
        return _at(g, "g", (H,), torch.float32, dev), 1
    return _at(g, "g", (B, L, H), torch.float32, dev), 0


def _scratch(workspace, need, dev):
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, device=dev, dtype=torch.uint8)
        return workspace.data_ptr(), need
    _req(workspace, "workspace", device=dev)  # (the library checks its size and alignment)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def linattn_fwd(q, k, v, g, h0=None, scale=None, lengths=None, want_ckpt: bool = True, want_h_last: bool = True,
                workspace=None):
    """Linear attention with a decay for each head -> ``(o, ckpt, h_last)``:
    ``S_t = exp(g_t) S_{t-1} + k_t v_t^T``, ``o_t = scale * S_t^T q_t`` from ``S = h0``.

    ``q, k`` [B, L, G, K] are shared by the H/G heads of a group of ``v`` [B, L, H, V]; each may be a column range of
    a wider [B, L, W] tensor.  ``g`` are log decays, fp32 [B, L, H] or one for each head [H].  ``lengths`` (int32 [B])
    ends each row; past it o is 0 and the state stays.  ``scale`` is ``K ** -0.5`` unless given.  ``ckpt`` (None unless
    ``want_ckpt``) is what ``linattn_bwd`` starts from.

    A NaN or infinity in a live token can reach the other tokens of its chunk (64 in fp32, 128 in bf16), also earlier ones."""
    B, L, H, G, K, V = _linattn_sizes(q, v)
    dev, dt, f32 = q.device, q.dtype, torch.float32
    sdt = _act_dtype(q)
    pq, ldq = _rows(q, "q", (B, L, G, K), dt, dev)
    pk, ldk = _rows(k, "k", (B, L, G, K), dt, dev)
    pv, ldv = _rows(v, "v", (B, L, H, V), dt, dev)
    pg, per_head = _linattn_gate(g, B, L, H, dev)
    ph = _opt_at(h0, "h0", (B, H, K, V), f32, dev)
    pn = _opt_at(lengths, "lengths", (B,), torch.int32, dev)
    chunks, need, _ = _linattn_plan(B, L, H, G, K, V, 0, sdt)
    o = torch.empty((B, L, H, V), device=dev, dtype=dt)
    ckpt = torch.empty((B, H, chunks, K, V), device=dev, dtype=f32) if want_ckpt else None
    h_last = torch.empty((B, H, K, V), device=dev, dtype=f32) if want_h_last else None
    pw, have = _scratch(workspace, need, dev)
    rc = load().linattn_fwd(pq, ldq, pk, ldk, pv, ldv, pg, per_head, ph, pn, o.data_ptr(),
                            ckpt.data_ptr() if want_ckpt else None, h_last.data_ptr() if want_h_last else None, B, L, H, G, K, V,
                            K ** -0.5 if scale is None else scale, sdt, pw, have, _raw_stream(dev))
    if rc:
        check(rc, "linattn_fwd")
    return o, ckpt, h_last


def linattn_bwd(q, k, v, g, ckpt, do, dh_last=None, scale=None, lengths=None, dg=None, want_dh0: bool = True,
                workspace=None):
    """Gradients of ``sum(o * do)`` (+ ``sum(h_last * dh_last)``) through ``linattn_fwd`` called with the same q, k, v, g,
    scale and lengths -> dict ``dq, dk, dv`` (q's type), ``dg``, ``dh0`` (fp32).  With one decay for each head ``dg`` [H]
    accumulates into the given tensor (zeros when None)."""
    B, L, H, G, K, V = _linattn_sizes(q, v)
    dev, dt, f32 = q.device, q.dtype, torch.float32
    sdt = _act_dtype(q)
    pq, ldq = _rows(q, "q", (B, L, G, K), dt, dev)
    pk, ldk = _rows(k, "k", (B, L, G, K), dt, dev)
    pv, ldv = _rows(v, "v", (B, L, H, V), dt, dev)
    pg, per_head = _linattn_gate(g, B, L, H, dev)
    chunks, _, need = _linattn_plan(B, L, H, G, K, V, per_head, sdt)
    pc = _at(ckpt, "ckpt", (B, H, chunks, K, V), f32, dev)
    pd = _at(do, "do", (B, L, H, V), dt, dev)
    pl = _opt_at(dh_last, "dh_last", (B, H, K, V), f32, dev)
    pn = _opt_at(lengths, "lengths", (B,), torch.int32, dev)
    if dg is None:
        dg = torch.zeros((H,), device=dev, dtype=f32) if per_head else torch.empty((B, L, H), device=dev, dtype=f32)
    dq = torch.empty((B, L, G, K), device=dev, dtype=dt)
    dk = torch.empty((B, L, G, K), device=dev, dtype=dt)
    dv = torch.empty((B, L, H, V), device=dev, dtype=dt)
    dh0 = torch.empty((B, H, K, V), device=dev, dtype=f32) if want_dh0 else None
    pw, have = _scratch(workspace, need, dev)
    rc = load().linattn_bwd(pq, ldq, pk, ldk, pv, ldv, pg, per_head, pn, pc, pd, pl, dq.data_ptr(), dk.data_ptr(),
                            dv.data_ptr(), _at(dg, "dg", g.shape, f32, dev), dh0.data_ptr() if want_dh0 else None, B, L, H, G, K, V,
                            K ** -0.5 if scale is None else scale, sdt, pw, have, _raw_stream(dev))
    if rc:
        check(rc, "linattn_bwd")
    return {"dq": dq, "dk": dk, "dv": dv, "dg": dg, "dh0": dh0}


def linattn_step(q, k, v, g, h, scale=None):
    """One token for B sequences: updates ``h`` [B, H, K, V] in place and returns o [B, H, V].
    ``q, k`` [B, G, K], ``v`` [B, H, V], ``g`` fp32 [B, H] or [H]."""
    B, G, K = q.shape
    _, H, V = v.shape
    dev, dt, f32 = q.device, q.dtype, torch.float32
    sdt = _act_dtype(q)
    pq, pk = _at(q, "q", (B, G, K), dt, dev), _at(k, "k", (B, G, K), dt, dev)
    pv, ph = _at(v, "v", (B, H, V), dt, dev), _at(h, "h", (B, H, K, V), f32, dev)
    per_head = 1 if g.dim() == 1 else 0
    pg = _at(g, "g", (H,) if per_head else (B, H), f32, dev)
    o = torch.empty_like(v)
    rc = load().linattn_step(pq, pk, pv, pg, per_head, ph, o.data_ptr(), B, H, G, K, V, K ** -0.5 if scale is None else scale,
                             sdt, _raw_stream(dev))
    if rc:
        check(rc, "linattn_step")
    return o


def layernorm_fwd(x, scale, bias, eps: float, want_stats: bool = True):
    """Layer norm of the rows of x [rows, dim]: ``(y, mean, rstd)`` with y in x's dtype and the statistics fp32 (None
    unless ``want_stats``); ``bias`` may be None."""
    R, N = x.shape
    dev, f32 = x.device, torch.float32
    dt = _act_dtype(x)
    px, ps = _at(x, "x", (R, N), x.dtype, dev), _at(scale, "scale", (N,), f32, dev)
    pb = _opt_at(bias, "bias", (N,), f32, dev)
    y = torch.empty_like(x)
    mean = torch.empty((R,), device=dev, dtype=f32) if want_stats else None
    rstd = torch.empty((R,), device=dev, dtype=f32) if want_stats else None
    rc = load().layernorm_fwd(px, ps, pb, eps, y.data_ptr(), mean.data_ptr() if want_stats else None,
                              rstd.data_ptr() if want_stats else None, R, N, dt, _raw_stream(dev))
    if rc:
        check(rc, "layernorm_fwd")
    return y, mean, rstd


def layernorm_bwd(dy, x, scale, mean, rstd, dscale=None, dbias=None, workspace=None):
    """Layer norm backward -> ``(dx, dscale, dbias)``, all fp32; dscale and dbias accumulate into the given tensors
    and are made when None."""
    R, N = x.shape
    dev, f32 = x.device, torch.float32
    dt = _act_dtype(x)
    py, px = _at(dy, "dy", (R, N), x.dtype, dev), _at(x, "x", (R, N), x.dtype, dev)
    ps = _at(scale, "scale", (N,), f32, dev)
    pm, pr = _at(mean, "mean", (R,), f32, dev), _at(rstd, "rstd", (R,), f32, dev)
    add = (1 if dscale is not None else 0) | (2 if dbias is not None else 0)
    if dscale is None:
        dscale = torch.empty((N,), device=dev, dtype=f32)
    if dbias is None:
        dbias = torch.empty((N,), device=dev, dtype=f32)
    dx = torch.empty((R, N), device=dev, dtype=f32)
    pw, have = _scratch(workspace, _layernorm_plan(R, N), dev)
    rc = load().layernorm_bwd(py, px, ps, pm, pr, dx.data_ptr(), _at(dscale, "dscale", (N,), f32, dev),
                              _at(dbias, "dbias", (N,), f32, dev), add, R, N, dt, pw, have, _raw_stream(dev))
    if rc:
        check(rc, "layernorm_bwd")
    return dx, dscale, dbias


def count_nonfinite(t, workspace=None) -> int:
    """Number of NaN / +-Inf values in a dense fp32 or bf16 CUDA tensor (synchronises the current stream)."""
    lib = load()
    dt = _act_dtype(t)
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("count_nonfinite: t must be a contiguous CUDA tensor")
    wsz = lib.ss_count_nonfinite_workspace_size()
    ws = workspace if workspace is not None else torch.empty((wsz,), device=t.device, dtype=torch.uint8)
    out = torch.empty((1,), device=t.device, dtype=torch.int64)
    rc = lib.ss_count_nonfinite(_p(t), t.numel(), dt, _p(out), _p(ws), ws.numel() * ws.element_size(), _stream())
    check(rc, "ss_count_nonfinite")
    return int(out.item())


def device_status() -> int:
    """Reads and clears the library's device error word (synchronises the current stream)."""
    return load().ss_device_status(_stream())
