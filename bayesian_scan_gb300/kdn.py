"""Thin ctypes binding of the C ABI in ``include/kdn.h``.

Argument marshalling only: every step of both scans runs in the CUDA
kernels of ``_build/libkdn.so``.  PyTorch provides device memory and the
current stream.  There is no CPU fallback: if the library is missing the
import of this module raises.

Functions mirror the C names:

* :func:`diag_scan_fwd`  -> ``kdn_diag_scan_fwd``
* :func:`diag_mobius_scan_fwd` -> ``kdn_diag_mobius_scan_fwd`` (per-head lambda in the same launch)
* :func:`mobius_scan`    -> ``kdn_mobius_scan``
* :func:`mobius_scan_noalloc` -> ``kdn_mobius_scan_noalloc``
* :func:`gated_scan_fwd`, :func:`gated_scan_bwd`, :func:`gated_step` -> ``kdn_gated_*`` (the
  recurrence with one gate per channel)
* :func:`qk_norm_rope_fwd`, :func:`qk_norm_rope_bwd` -> ``kdn_qk_norm_rope_*`` (queries and keys for
  the scans)
* :func:`delta_scan_fwd`, :func:`delta_scan_bwd`, :func:`delta_step` -> ``kdn_delta_*`` (the gated
  delta rule)
* :func:`add_rms_norm_fwd`, :func:`add_rms_norm_bwd` -> ``kdn_add_rms_norm_*`` (the residual's addition
  and its norm)
* :func:`diag_scan_plan`, :func:`mobius_scan_plan` -> the ``*_plan`` queries
* :func:`get_device_error`, :func:`set_wait_limit_ns`,
  :func:`debug_stall_mobius_tile`, :func:`debug_stall_gated_rank`,
  :func:`debug_stall_delta_chunk`, :func:`status_string`,
  :func:`version`

When the tensors passed to :func:`diag_scan_fwd` / :func:`mobius_scan` live in
host memory, the call stages them to the current device on the current stream
(pinned memory makes the copies asynchronous), runs the kernels there and
copies the results back; it returns host tensors.

Every call is issued on torch's current stream, or on ``stream``.  Given one,
the call's inputs have to be ready there, and what it allocates (outputs and
workspaces) is that stream's memory, as under ``torch.cuda.stream(stream)``.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os

import torch

from . import build as _build

KDN_OK, KDN_ERR_INVALID_ARG, KDN_ERR_UNSUPPORTED = 0, -1, -2
KDN_ERR_CUDA, KDN_ERR_TIMEOUT, KDN_ERR_ALLOC = -3, -4, -5
KDN_F32, KDN_BF16, KDN_E4M3 = 0, 1, 2

LIB_PATH = _build.LIB


class KdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libkdn is not built ({LIB_PATH}); run bayesian_scan_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fp, i, ll = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
    lib.kdn_diag_scan_fwd.restype = i
    lib.kdn_diag_scan_fwd.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, fp, fp, fp, fp,
                                      i, i, i, i, i, i, vp]
    lib.kdn_mobius_scan.restype = i
    lib.kdn_mobius_scan.argtypes = [fp, fp, fp, fp, fp, fp, ll, ll, vp]
    lib.kdn_diag_mobius_scan_fwd.restype = i
    lib.kdn_diag_mobius_scan_fwd.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, fp, fp, fp, fp,
                                             fp, fp, fp, fp, fp, fp, i, i, i, i, i, i, vp]
    lib.kdn_lin_scan_fwd.restype = i
    lib.kdn_lin_scan_fwd.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, fp, fp, fp,
                                     i, i, i, i, i, i, vp]
    lib.kdn_diag_scan_bwd.restype = i
    lib.kdn_diag_scan_bwd.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, fp, fp, fp, fp,
                                      fp, fp, fp, fp, fp, fp, fp, i, i, i, i, i, i, vp, ll, vp]
    lib.kdn_diag_scan_bwd_workspace.restype = i
    lib.kdn_diag_scan_bwd_workspace.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_longlong)]
    lib.kdn_diag_step.restype = i
    lib.kdn_diag_step.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, fp, fp, i, i, i, i, i, vp]
    lib.kdn_diag_scan_fwd_host.restype = i
    lib.kdn_diag_scan_fwd_host.argtypes = [vp, vp, vp, vp, vp, fp, ctypes.c_float, fp, fp, fp, fp,
                                           i, i, i, i, i, i, vp]
    lib.kdn_mobius_scan_host.restype = i
    lib.kdn_mobius_scan_host.argtypes = [fp, fp, fp, fp, fp, fp, ll, ll, vp]
    lib.kdn_mobius_scan_noalloc.restype = i
    lib.kdn_mobius_scan_noalloc.argtypes = [fp, fp, fp, fp, fp, fp, ll, ll, vp]
    lib.kdn_gated_scan_fwd.restype = i
    lib.kdn_gated_scan_fwd.argtypes = [vp, ll, vp, ll, fp, fp, vp, i, i, vp, fp, i, i, i, i, i, i, vp]
    lib.kdn_gated_scan_bwd.restype = i
    lib.kdn_gated_scan_bwd.argtypes = [vp, ll, vp, ll, fp, fp, vp, i, i, vp, vp, fp, vp, vp, fp, fp,
                                       i, i, i, i, i, i, vp, ll, vp]
    lib.kdn_gated_scan_bwd_workspace.restype = i
    lib.kdn_gated_scan_bwd_workspace.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_longlong)]
    lib.kdn_gated_step.restype = i
    lib.kdn_gated_step.argtypes = [vp, vp, fp, i, fp, fp, vp, i, i, i, i, i, vp]
    lib.kdn_qk_norm_rope_fwd.restype = i
    lib.kdn_qk_norm_rope_fwd.argtypes = [vp, ll, vp, ll, fp, fp, i, ctypes.c_float, vp, i, fp, vp, i, i,
                                         vp, vp, i, i, i, i, i, i, i, vp]
    lib.kdn_qk_norm_rope_bwd.restype = i
    lib.kdn_qk_norm_rope_bwd.argtypes = [vp, ll, vp, ll, fp, fp, i, ctypes.c_float, vp, i, fp, vp, i, i,
                                         vp, vp, vp, ll, vp, ll, fp, fp, i, i, i, i, i, i, i, vp, ll, vp]
    lib.kdn_qk_norm_rope_bwd_workspace.restype = i
    lib.kdn_qk_norm_rope_bwd_workspace.argtypes = [i, i, i, i, i, ctypes.POINTER(ctypes.c_longlong)]
    lib.kdn_delta_scan_fwd.restype = i
    lib.kdn_delta_scan_fwd.argtypes = [vp, vp, vp, vp, vp, fp, fp, vp, i, vp, fp, i, i, i, i, i, i, i, vp, ll, vp]
    lib.kdn_delta_scan_bwd.restype = i
    lib.kdn_delta_scan_bwd.argtypes = [vp, vp, vp, vp, vp, fp, fp, vp, i, vp, fp, vp, vp, vp, vp, vp, fp, fp,
                                       i, i, i, i, i, i, i, vp, ll, vp]
    for f in (lib.kdn_delta_scan_fwd_workspace, lib.kdn_delta_scan_bwd_workspace):
        f.restype = i
        f.argtypes = [i, i, i, i, i, i, i, ctypes.POINTER(ctypes.c_longlong)]
    lib.kdn_delta_step.restype = i
    lib.kdn_delta_step.argtypes = [vp, vp, vp, vp, vp, fp, fp, fp, vp, i, i, i, i, i, i, vp]
    lib.kdn_add_rms_norm_fwd.restype = i
    lib.kdn_add_rms_norm_fwd.argtypes = [vp, ll, vp, fp, ctypes.c_float, vp, vp, fp, ll, i, i, i, i, vp]
    lib.kdn_add_rms_norm_bwd.restype = i
    lib.kdn_add_rms_norm_bwd.argtypes = [vp, fp, ctypes.c_float, vp, vp, vp, vp, fp, ll, i, i, i, i, vp, ll, vp]
    lib.kdn_add_rms_norm_bwd_workspace.restype = i
    lib.kdn_add_rms_norm_bwd_workspace.argtypes = [ll, i, ctypes.POINTER(ctypes.c_longlong)]
    lib.kdn_status_string.restype = ctypes.c_char_p
    lib.kdn_status_string.argtypes = [i]
    lib.kdn_get_device_error.restype = i
    lib.kdn_get_device_error.argtypes = [vp]
    lib.kdn_set_wait_limit_ns.restype = None
    lib.kdn_set_wait_limit_ns.argtypes = [ll]
    lib.kdn_debug_stall_mobius_tile.restype = None
    lib.kdn_debug_stall_mobius_tile.argtypes = [ll]
    lib.kdn_debug_stall_gated_rank.restype = None
    lib.kdn_debug_stall_gated_rank.argtypes = [i]
    lib.kdn_debug_stall_delta_chunk.restype = None
    lib.kdn_debug_stall_delta_chunk.argtypes = [i]
    ip, llp = ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_longlong)
    lib.kdn_diag_scan_plan.restype = i
    lib.kdn_diag_scan_plan.argtypes = [i, i, i, i, i, i, ip, ip, llp]
    lib.kdn_mobius_scan_plan.restype = i
    lib.kdn_mobius_scan_plan.argtypes = [ll, ll, ip, llp]
    lib.kdn_version.restype = ctypes.c_char_p
    lib.kdn_version.argtypes = []
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.kdn_status_string(int(status)).decode()


def version() -> str:
    return lib.kdn_version().decode()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    # the raw handle of torch's current stream: a stream object costs as much
    # host time as the rest of a small call
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _alloc(stream):
    """Where a call makes the tensors that its caller did not give: in the
    memory of the stream that will write them.  (A block that another stream
    has let go may still be read by work queued there.)"""
    if stream is None:
        return _CURRENT
    return torch.cuda.stream(stream if hasattr(stream, "device") else torch.cuda.ExternalStream(stream.cuda_stream))


_CURRENT = contextlib.nullcontext()


def _check(t, name, dtype=None, shape=None):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _check_workspace(t, nbytes):
    _check(t, "workspace")
    if t.numel() * t.element_size() < nbytes:
        raise ValueError(f"workspace must hold {nbytes} bytes")


def _on_one_device(stream, **tensors):
    """Every given tensor must be a CUDA tensor on the current device (the
    device whose stream the call is issued on): the C ABI receives raw
    pointers and cannot tell host memory or another GPU's memory apart."""
    seen = {t.get_device() for t in tensors.values() if t is not None}
    if stream is None and len(seen) == 1 and min(seen) >= 0 and torch._C._cuda_getDevice() in seen:
        return
    given = [(name, t) for name, t in tensors.items() if t is not None]
    for name, t in given:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the call takes device tensors)")
    cur = torch.device("cuda", torch.cuda.current_device())
    for name, t in given:
        if t.device != cur:
            raise ValueError(f"{name} is on {t.device} but the current device is {cur}")
    if stream is not None and getattr(stream, "device", cur) != cur:
        raise ValueError(f"the stream belongs to {stream.device}, not the current device {cur}")


def diag_scan_fwd(q, k, v, beta, d, A, I_prior=1.0, I0=None, mu0=None, out=None,
                  final_state=True, stream=None):
    """Diagonal metaplastic scan with readout (see ``kdn_diag_scan_fwd``).

    q, k [B,H,T,dk]; v, beta [B,H,T,dv]; d [B,H,T] (bf16 or fp32, all the same);
    A [H] fp32; I0, mu0 [B,H,dv,dk] fp32 or None.  ``final_state`` may be
    True (allocate), False/None (skip) or a [2,B,H,dv,dk] fp32 tensor.
    Returns (out [B,H,T,dv] fp32, final_state or None).  With host tensors
    the call goes to ``kdn_diag_scan_fwd_host`` (pipelined copies; outputs
    are host tensors, page-locked when allocated here).
    """
    if not q.is_cuda:
        return _diag_host(q, k, v, beta, d, A, I_prior, I0, mu0, out, final_state, stream)
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bf16 or fp32")
    _check(q, "q", dt)
    _check(k, "k", dt, (B, H, T, dk))
    _check(v, "v", dt, (B, H, T, dv))
    _check(beta, "beta", dt, (B, H, T, dv))
    _check(d, "d", dt, (B, H, T))
    _check(A, "A", torch.float32, (H,))
    for name, t in (("I0", I0), ("mu0", mu0)):
        if t is not None:
            _check(t, name, torch.float32, (B, H, dv, dk))
    if out is None:
        with _alloc(stream):
            out = torch.empty(B, H, T, dv, device=q.device, dtype=torch.float32)
    _check(out, "out", torch.float32, (B, H, T, dv))
    if final_state is True:
        with _alloc(stream):
            final_state = torch.empty(2, B, H, dv, dk, device=q.device, dtype=torch.float32)
    elif final_state is False:
        final_state = None
    if final_state is not None:
        _check(final_state, "final_state", torch.float32, (2, B, H, dv, dk))
    _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, I0=I0, mu0=mu0, out=out,
                   final_state=final_state)
    st = lib.kdn_diag_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A),
                               float(I_prior), _ptr(I0), _ptr(mu0), _ptr(out), _ptr(final_state),
                               B, H, T, dk, dv, KDN_BF16 if dt == torch.bfloat16 else KDN_F32,
                               _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_scan_fwd")
    return out, final_state


def diag_mobius_scan_fwd(q, k, v, beta, d, A, ma, mb, mc, md, lambda0, I_prior=1.0, I0=None,
                         mu0=None, out=None, final_state=True, lambda_out=None, stream=None):
    """The diagonal scan and the per-head Moebius scan in one launch (see
    ``kdn_diag_mobius_scan_fwd``).  Diagonal-scan arguments as for
    ``diag_scan_fwd`` (device tensors); ma, mb, mc, md [B*H,T] fp32 (row b*H +
    h), lambda0 [B*H] fp32.  Returns (out, final_state or None, lambda
    [B*H,T])."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bf16 or fp32")
    _check(q, "q", dt)
    _check(k, "k", dt, (B, H, T, dk))
    _check(v, "v", dt, (B, H, T, dv))
    _check(beta, "beta", dt, (B, H, T, dv))
    _check(d, "d", dt, (B, H, T))
    _check(A, "A", torch.float32, (H,))
    for name, t in (("I0", I0), ("mu0", mu0)):
        if t is not None:
            _check(t, name, torch.float32, (B, H, dv, dk))
    for name, t in (("ma", ma), ("mb", mb), ("mc", mc), ("md", md)):
        _check(t, name, torch.float32, (B * H, T))
    _check(lambda0, "lambda0", torch.float32, (B * H,))
    _on_one_device(stream, q=q)
    if out is None:
        with _alloc(stream):
            out = torch.empty(B, H, T, dv, device=q.device, dtype=torch.float32)
    _check(out, "out", torch.float32, (B, H, T, dv))
    if final_state is True:
        with _alloc(stream):
            final_state = torch.empty(2, B, H, dv, dk, device=q.device, dtype=torch.float32)
    elif final_state is False:
        final_state = None
    if final_state is not None:
        _check(final_state, "final_state", torch.float32, (2, B, H, dv, dk))
    if lambda_out is None:
        with _alloc(stream):
            lambda_out = torch.empty(B * H, T, device=q.device, dtype=torch.float32)
    _check(lambda_out, "lambda_out", torch.float32, (B * H, T))
    _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, I0=I0, mu0=mu0, out=out,
                   final_state=final_state, ma=ma, mb=mb, mc=mc, md=md, lambda0=lambda0,
                   lambda_out=lambda_out)
    st = lib.kdn_diag_mobius_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A),
                                      float(I_prior), _ptr(I0), _ptr(mu0), _ptr(out),
                                      _ptr(final_state), _ptr(ma), _ptr(mb), _ptr(mc), _ptr(md),
                                      _ptr(lambda0), _ptr(lambda_out), B, H, T, dk, dv,
                                      KDN_BF16 if dt == torch.bfloat16 else KDN_F32, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_mobius_scan_fwd")
    return out, final_state, lambda_out


def lin_scan_fwd(q, k, v, beta, d, A, I_prior=1.0, mu0=None, out=None, final_mu=True,
                 stream=None):
    """The non-metaplastic limit (importance held at I_prior; see
    ``kdn_lin_scan_fwd``).  Device tensors as for ``diag_scan_fwd``; mu0
    [B,H,dv,dk] fp32 or None; ``final_mu`` True (allocate), False/None or a
    [B,H,dv,dk] fp32 tensor.  Returns (out, final_mu or None)."""
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bf16 or fp32")
    if not q.is_cuda:
        raise ValueError("lin_scan_fwd takes device tensors")
    _check(q, "q", dt)
    _check(k, "k", dt, (B, H, T, dk))
    _check(v, "v", dt, (B, H, T, dv))
    _check(beta, "beta", dt, (B, H, T, dv))
    _check(d, "d", dt, (B, H, T))
    _check(A, "A", torch.float32, (H,))
    if mu0 is not None:
        _check(mu0, "mu0", torch.float32, (B, H, dv, dk))
    if out is None:
        with _alloc(stream):
            out = torch.empty(B, H, T, dv, device=q.device, dtype=torch.float32)
    _check(out, "out", torch.float32, (B, H, T, dv))
    if final_mu is True:
        with _alloc(stream):
            final_mu = torch.empty(B, H, dv, dk, device=q.device, dtype=torch.float32)
    elif final_mu is False:
        final_mu = None
    if final_mu is not None:
        _check(final_mu, "final_mu", torch.float32, (B, H, dv, dk))
    _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, mu0=mu0, out=out, final_mu=final_mu)
    st = lib.kdn_lin_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A),
                              float(I_prior), _ptr(mu0), _ptr(out), _ptr(final_mu),
                              B, H, T, dk, dv, KDN_BF16 if dt == torch.bfloat16 else KDN_F32,
                              _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_lin_scan_fwd")
    return out, final_mu


def diag_scan_bwd_workspace(B, H, T, dk, dv) -> int:
    """Bytes of device workspace ``diag_scan_bwd`` needs."""
    n = ctypes.c_longlong(0)
    st = lib.kdn_diag_scan_bwd_workspace(B, H, T, dk, dv, ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_scan_bwd_workspace")
    return int(n.value)


def diag_scan_bwd(q, k, v, beta, d, A, grad_out, I_prior=1.0, I0=None, mu0=None,
                  grad_final_state=None, grad_init_state=True, workspace=None, stream=None):
    """Backward pass of ``diag_scan_fwd`` (see ``kdn_diag_scan_bwd``).

    Inputs as for ``diag_scan_fwd`` (device tensors); ``grad_out`` [B,H,T,dv]
    fp32; ``grad_final_state`` [2,B,H,dv,dk] fp32 or None.  ``grad_init_state``
    True (allocate), False/None (skip) or a [2,B,H,dv,dk] fp32 tensor.
    Returns a dict: q, k [B,H,T,dk]; v, beta [B,H,T,dv]; d [B,H,T]; A [H];
    init_state [2,B,H,dv,dk] or None (all fp32).  ``workspace``: a uint8
    device tensor of at least ``diag_scan_bwd_workspace`` bytes, or None (one
    is taken from torch's caching allocator for the call).
    """
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bf16 or fp32")
    if not q.is_cuda:
        raise ValueError("diag_scan_bwd takes device tensors")
    _check(q, "q", dt)
    _check(k, "k", dt, (B, H, T, dk))
    _check(v, "v", dt, (B, H, T, dv))
    _check(beta, "beta", dt, (B, H, T, dv))
    _check(d, "d", dt, (B, H, T))
    _check(A, "A", torch.float32, (H,))
    _check(grad_out, "grad_out", torch.float32, (B, H, T, dv))
    for name, t in (("I0", I0), ("mu0", mu0)):
        if t is not None:
            _check(t, name, torch.float32, (B, H, dv, dk))
    if grad_final_state is not None:
        _check(grad_final_state, "grad_final_state", torch.float32, (2, B, H, dv, dk))
    f32 = dict(device=q.device, dtype=torch.float32)
    with _alloc(stream):
        g = dict(q=torch.empty(B, H, T, dk, **f32), k=torch.empty(B, H, T, dk, **f32),
                 v=torch.empty(B, H, T, dv, **f32), beta=torch.empty(B, H, T, dv, **f32),
                 d=torch.empty(B, H, T, **f32), A=torch.empty(H, **f32))
    if grad_init_state is True:
        with _alloc(stream):
            grad_init_state = torch.empty(2, B, H, dv, dk, **f32)
    elif grad_init_state is False:
        grad_init_state = None
    if grad_init_state is not None:
        _check(grad_init_state, "grad_init_state", torch.float32, (2, B, H, dv, dk))
    g["init_state"] = grad_init_state
    ws_bytes = diag_scan_bwd_workspace(B, H, T, dk, dv)
    if workspace is None:
        with _alloc(stream):
            workspace = torch.empty(max(ws_bytes, 1), device=q.device, dtype=torch.uint8)
    else:
        _check_workspace(workspace, ws_bytes)
    _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, I0=I0, mu0=mu0, grad_out=grad_out,
                   grad_final_state=grad_final_state, grad_init_state=grad_init_state,
                   workspace=workspace)
    st = lib.kdn_diag_scan_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A),
                               float(I_prior), _ptr(I0), _ptr(mu0), _ptr(grad_out),
                               _ptr(grad_final_state), _ptr(g["q"]), _ptr(g["k"]), _ptr(g["v"]),
                               _ptr(g["beta"]), _ptr(g["d"]), _ptr(g["A"]), _ptr(grad_init_state),
                               B, H, T, dk, dv, KDN_BF16 if dt == torch.bfloat16 else KDN_F32,
                               _ptr(workspace), ws_bytes, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_scan_bwd")
    return g


def diag_step(q, k, v, beta, d, A, state, I_prior=1.0, out=None, stream=None):
    """One token of the diagonal update on a device-resident state (see
    ``kdn_diag_step``): q, k [B,H,dk]; v, beta [B,H,dv]; d [B,H] (bf16 or
    fp32); A [H] fp32; state [2,B,H,dv,dk] fp32 (mu then I), updated in place.
    Returns out [B,H,dv] fp32."""
    B, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bf16 or fp32")
    for name, t, shape, dtype in (("q", q, (B, H, dk), dt), ("k", k, (B, H, dk), dt),
                                  ("v", v, (B, H, dv), dt), ("beta", beta, (B, H, dv), dt),
                                  ("d", d, (B, H), dt), ("A", A, (H,), torch.float32),
                                  ("state", state, (2, B, H, dv, dk), torch.float32)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        _check(t, name, dtype, shape)
    if out is None:
        with _alloc(stream):
            out = torch.empty(B, H, dv, device=q.device, dtype=torch.float32)
    _check(out, "out", torch.float32, (B, H, dv))
    _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, state=state, out=out)
    st = lib.kdn_diag_step(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A), float(I_prior),
                           _ptr(state), _ptr(out), B, H, dk, dv,
                           KDN_BF16 if dt == torch.bfloat16 else KDN_F32, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_step")
    return out


def mobius_scan(a, b, c, d, lambda0, out=None, stream=None):
    """Moebius precision recursion (see ``kdn_mobius_scan``): a,b,c,d [N,T]
    fp32, lambda0 [N] fp32 -> lambda_1..lambda_T [N,T] fp32.  Host tensors go
    to ``kdn_mobius_scan_host``."""
    if not a.is_cuda:
        return _mobius_host(a, b, c, d, lambda0, out, stream)
    N, T = a.shape
    for name, t in (("a", a), ("b", b), ("c", c), ("d", d)):
        _check(t, name, torch.float32, (N, T))
    _check(lambda0, "lambda0", torch.float32, (N,))
    if out is None:
        with _alloc(stream):
            out = torch.empty(N, T, device=a.device, dtype=torch.float32)
    _check(out, "out", torch.float32, (N, T))
    _on_one_device(stream, a=a, b=b, c=c, d=d, lambda0=lambda0, out=out)
    st = lib.kdn_mobius_scan(_ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(lambda0), _ptr(out),
                             N, T, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_mobius_scan")
    return out


# ---------------------------------------------------------------------------
# the recurrence with one gate per channel

def _here(stream, *tensors):
    """Whether the given tensors (None: not given) are all on the current
    device and the call goes to its current stream; where not,
    ``_on_one_device`` has the message."""
    if stream is not None:
        return False
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if dev is not None:
                    return False
                dev = d
    return dev is not None and dev >= 0 and dev == torch._C._cuda_getDevice()


_DTYPES = {torch.bfloat16: KDN_BF16, torch.float32: KDN_F32}
_F32 = torch.float32


def _new(like, dtype, stream):
    """An uninitialised dense tensor of like's shape."""
    if stream is not None:
        with _alloc(stream):
            return _new(like, dtype, None)
    if dtype is None or dtype is like.dtype:
        if like.is_contiguous():
            return torch.empty_like(like)
        dtype = like.dtype
    return torch.empty(like.shape, device=like.device, dtype=dtype)


def _dtype_of(t, name):
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise ValueError(f"{name} must be bf16 or fp32, got {t.dtype}")
    return dt


def _ws_device(t):
    """The device a workspace size is asked for, the current one: the size is
    a matter of its SMs, and a call on another device's tensors is refused."""
    return torch._C._cuda_getDevice() if t.is_cuda else -1


def _scratch(nbytes, like, stream):
    """A call's own workspace, let go when the call returns: the stream's next
    allocations may have it, in the stream's order."""
    return _empty(nbytes, like, torch.uint8, stream)


_MOST = 0x7fffffff


def _ints(*sizes):
    """The C calls take sizes of 32 bits, to which ctypes cuts larger ones
    without a word."""
    if max(sizes) > _MOST:
        raise ValueError(f"sizes must be below 2**31, got {sizes}")


def _empty(shape, like, dtype, stream):
    """An uninitialised tensor on like's device, the stream's memory."""
    if stream is not None:
        with _alloc(stream):
            return torch.empty(shape, device=like.device, dtype=dtype)
    return torch.empty(shape, device=like.device, dtype=dtype)


def _dense_like(t, stream):
    """The same of t's shape and type; ``torch.empty_like`` where there is no
    stream and t is dense."""
    with _alloc(stream):
        return torch.empty_like(t, memory_format=torch.contiguous_format)


def _token_ld(t, name, dt, shape):
    """Elements between consecutive tokens of a [B,T,C] or [B,H,T,C] tensor
    whose channels are adjacent and whose rows follow one another (dense, or
    for one head a column slice of a wider projection)."""
    if t.dtype != dt:
        raise ValueError(f"{name} must be {dt}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    T, C = shape[-2], shape[-1]
    if t.is_contiguous():
        return C
    st = t.stride()
    ld = st[-2] if T > 1 else (st[0] if shape[0] > 1 and len(shape) == 3 else C)
    if (C > 1 and st[-1] != 1) or ld < C:
        raise ValueError(f"{name} must have adjacent channels and tokens apart by at least their number")
    step = T * ld
    for n, s in zip(reversed(shape[:-2]), reversed(st[:-2])):
        if n > 1 and s != step:
            raise ValueError(f"{name}'s rows must follow one another (stride {step}), got stride {s}")
        step *= n
    return ld


def _gated_sizes(x, A, offsets):
    """(B, H, T, C, state rows, their shape) of a gated-recurrence call."""
    if x.dim() == 3:
        (B, T, C), H = x.shape, 1
    elif x.dim() == 4:
        B, H, T, C = x.shape
    else:
        raise ValueError(f"x must be [B,T,C] or [B,H,T,C], got {tuple(x.shape)}")
    heads = (C,) if x.dim() == 3 else (H, C)
    _check(A, "A", torch.float32, heads)
    rows = B
    if offsets is not None:
        _check(offsets, "offsets", torch.int32)
        if offsets.dim() != 1 or offsets.numel() < 2 or B != 1:
            raise ValueError("offsets must be [nseq + 1] with B = 1")
        rows = offsets.numel() - 1
    if (B | H | T | C | rows) > _MOST:
        _ints(B, H, T, C, rows)
    return B, H, T, C, 0 if offsets is None else rows, (rows, *heads)


def gated_scan_fwd(x, d, A, h0=None, leak=False, offsets=None, out=None, out_dtype=None,
                   final_state=True, stream=None):
    """Gated recurrence h_t = alpha_t h_{t-1} + w_t x_t, alpha_t = exp(-A d_t),
    w_t = 1 or 1 - alpha_t with ``leak`` (see ``kdn_gated_scan_fwd``).

    x, d [B,T,C] with A [C], or [B,H,T,C] with A [H,C] (x, d bf16 or fp32,
    A fp32); a [B,T,C] x or d may be a column slice of a wider projection.
    h0 [B,(H,)C] fp32 or None.  ``offsets`` [nseq + 1] int32 (device): packed
    sequences in x [1,T,C] or [1,H,T,C]; h0 and final_state are then
    [nseq,(H,)C].  ``out_dtype`` is out's type (x's by default);
    ``final_state`` True (allocate), False/None (skip) or a tensor.  Returns
    (out, final_state or None).  With offsets, rows of an ``out`` allocated
    here that lie in no sequence are undefined."""
    B, H, T, C, nseq, state = _gated_sizes(x, A, offsets)
    it = _dtype_of(x, "x")
    x_ld = _token_ld(x, "x", x.dtype, x.shape)
    d_ld = _token_ld(d, "d", x.dtype, x.shape)
    if h0 is not None:
        _check(h0, "h0", torch.float32, state)
    if out is None:
        out = _new(x, out_dtype, stream)
    else:
        _check(out, "out", out_dtype, x.shape)
    ot = _dtype_of(out, "out")
    if final_state is True:
        final_state = _empty(state, x, _F32, stream)
    elif final_state is False:
        final_state = None
    elif final_state is not None:
        _check(final_state, "final_state", _F32, state)
    if not _here(stream, x, d, A, h0, offsets, out, final_state):
        _on_one_device(stream, x=x, d=d, A=A, h0=h0, offsets=offsets, out=out, final_state=final_state)
    st = lib.kdn_gated_scan_fwd(x.data_ptr(), x_ld, d.data_ptr(), d_ld, A.data_ptr(), _ptr(h0), _ptr(offsets), nseq,
                                int(leak), out.data_ptr(), _ptr(final_state), B, H, T, C, it, ot,
                                _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_gated_scan_fwd")
    return out, final_state


def gated_scan_bwd_workspace(B, H, T, C, nseq=0) -> int:
    """Bytes of device workspace ``gated_scan_bwd`` needs (0: none)."""
    _ints(B, H, T, C, nseq)
    n = ctypes.c_longlong(0)
    st = lib.kdn_gated_scan_bwd_workspace(B, H, T, C, nseq, ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, "kdn_gated_scan_bwd_workspace")
    return int(n.value)


@functools.lru_cache(maxsize=256)
def _gated_ws(device, B, H, T, C, nseq):
    return gated_scan_bwd_workspace(B, H, T, C, nseq)


def gated_scan_bwd(x, d, A, out, grad_out, h0=None, leak=False, offsets=None, grad_final_state=None,
                   grad_x=None, grad_d=None, grad_A=True, grad_h0=True, workspace=None, stream=None):
    """Backward pass of ``gated_scan_fwd`` (see ``kdn_gated_scan_bwd``): x, d,
    A, h0, leak and offsets as given to it, ``out`` its output, ``grad_out``
    of out's type.  ``grad_x``, ``grad_d``: dense tensors of x's type to write,
    or None (allocate); ``grad_A``, ``grad_h0``: True (allocate), False/None
    (skip) or fp32 tensors.  Returns a dict x, d, A, h0.  ``workspace``: a
    uint8 device tensor of at least ``gated_scan_bwd_workspace`` bytes, or
    None (one is taken from torch's caching allocator for the call)."""
    B, H, T, C, nseq, state = _gated_sizes(x, A, offsets)
    it = _dtype_of(x, "x")
    x_ld = _token_ld(x, "x", x.dtype, x.shape)
    d_ld = _token_ld(d, "d", x.dtype, x.shape)
    ot = _dtype_of(out, "out")
    _check(out, "out", None, x.shape)
    _check(grad_out, "grad_out", out.dtype, x.shape)
    for name, t in (("h0", h0), ("grad_final_state", grad_final_state)):
        if t is not None:
            _check(t, name, torch.float32, state)
    g = {}
    for name, t in (("x", grad_x), ("d", grad_d)):
        if t is None:
            t = _new(x, None, stream)
        else:
            _check(t, "grad_" + name, x.dtype, x.shape)
        g[name] = t
    for name, t, shape in (("A", grad_A, tuple(A.shape)), ("h0", grad_h0, state)):
        if t is True:
            like = A if name == "A" else h0
            t = (_empty(shape, x, _F32, stream) if like is None else
                 torch.empty_like(like) if stream is None else _dense_like(like, stream))
        elif t is False:
            t = None
        elif t is not None:
            _check(t, "grad_" + name, _F32, shape)
        g[name] = t
    ws_bytes = _gated_ws(_ws_device(x), B, H, T, C, nseq)
    if workspace is None:
        if ws_bytes:
            workspace = _scratch(ws_bytes, x, stream)
    else:
        _check_workspace(workspace, ws_bytes)
    gx, gd, gA, gh0 = g["x"], g["d"], g["A"], g["h0"]
    if not _here(stream, x, d, A, h0, offsets, out, grad_out, grad_final_state, gx, gd, gA, gh0, workspace):
        _on_one_device(stream, x=x, d=d, A=A, h0=h0, offsets=offsets, out=out, grad_out=grad_out,
                       grad_final_state=grad_final_state, grad_x=gx, grad_d=gd, grad_A=gA, grad_h0=gh0,
                       workspace=workspace)
    st = lib.kdn_gated_scan_bwd(x.data_ptr(), x_ld, d.data_ptr(), d_ld, A.data_ptr(), _ptr(h0), _ptr(offsets), nseq,
                                int(leak), out.data_ptr(), grad_out.data_ptr(), _ptr(grad_final_state),
                                gx.data_ptr(), gd.data_ptr(), _ptr(gA), _ptr(gh0), B, H, T, C,
                                it, ot, _ptr(workspace), ws_bytes, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_gated_scan_bwd")
    return g


def gated_step(x, d, A, state, leak=False, new_state=None, out=None, out_dtype=None, stream=None):
    """One token of ``gated_scan_fwd`` from a device-resident state (see
    ``kdn_gated_step``): x, d [B,C] with A [C], or [B,H,C] with A [H,C]; state
    fp32 of x's shape, updated in place, or left as it is when ``new_state``
    is another tensor to write.  Returns out (x's type unless ``out_dtype``
    says otherwise)."""
    shape, dt = x.shape, x.dtype
    if len(shape) not in (2, 3):
        raise ValueError(f"x must be [B,C] or [B,H,C], got {tuple(shape)}")
    if not 0 < x.numel() <= _MOST:                             # (else every size is below)
        _ints(*shape)
    it = _dtype_of(x, "x")
    if new_state is None:
        new_state = state
    if out is None:
        out = _new(x, out_dtype, stream)
    heads = shape[1:]
    # a step is a few microseconds: one expression where all is well, the
    # messages where it is not
    if not (d.dtype is dt and A.dtype is _F32 and state.dtype is _F32 and new_state.dtype is _F32
            and (out_dtype is None or out.dtype is out_dtype)
            and d.shape == shape and state.shape == shape and new_state.shape == shape and out.shape == shape
            and A.shape == heads and x.is_contiguous() and d.is_contiguous() and A.is_contiguous()
            and state.is_contiguous() and new_state.is_contiguous() and out.is_contiguous()):
        _check(x, "x")
        _check(d, "d", dt, shape)
        _check(A, "A", _F32, heads)
        _check(state, "state", _F32, shape)
        _check(new_state, "new_state", _F32, shape)
        _check(out, "out", out_dtype, shape)
    ot = _dtype_of(out, "out")
    if not _here(stream, x, d, A, state, new_state, out):
        _on_one_device(stream, x=x, d=d, A=A, state=state, new_state=new_state, out=out)
    st = lib.kdn_gated_step(x.data_ptr(), d.data_ptr(), A.data_ptr(), int(leak), state.data_ptr(),
                            new_state.data_ptr(), out.data_ptr(), shape[0], 1 if len(shape) == 2 else shape[1],
                            shape[-1], it, ot, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_gated_step")
    return out


# ---------------------------------------------------------------------------
# queries and keys for the scans

KDN_NORM_NONE, KDN_NORM_RMS, KDN_NORM_L2 = 0, 1, 2
_NORMS = {"none": KDN_NORM_NONE, "rms": KDN_NORM_RMS, "l2": KDN_NORM_L2}


def _head_rows(t, name, dt, B, T, dk):
    """(heads, elements between tokens) of a [B,T,H,dk] tensor whose heads lie
    side by side (dense, or a column slice of a fused projection)."""
    shape = t.shape
    if len(shape) != 4 or shape[0] != B or shape[1] != T or shape[3] != dk:
        raise ValueError(f"{name} must be [{B},{T},heads,{dk}], got {tuple(shape)}")
    if t.dtype != dt:
        raise ValueError(f"{name} must be {dt}, got {t.dtype}")
    H = shape[2]
    if (B | T | H | dk) > _MOST:
        _ints(B, T, H, dk)
    if t.is_contiguous():
        return H, H * dk
    st = t.stride()
    ld = st[1] if T > 1 else (st[0] if B > 1 else H * dk)
    if st[3] != 1 or (H > 1 and st[2] != dk) or ld < H * dk or (B > 1 and st[0] != T * ld):
        raise ValueError(f"{name}'s heads must lie side by side and its tokens be evenly apart")
    return H, ld


def _qk_common(q, k, pos, inv_freq, wq, wk, norm, axis):
    """Checks what the forward and the backward share; returns (B, T, dk,
    dtype, norm, axes, rot, (Hq, q_ld), (Hk, k_ld))."""
    first = q if q is not None else k
    if first is None:
        raise ValueError("q or k must be given")
    if first.dim() != 4:
        raise ValueError(f"q and k must be [B,T,H,dk], got {tuple(first.shape)}")
    B, T, _, dk = first.shape
    dtype = first.dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        _dtype_of(first, "q" if q is not None else "k")
    q_rows = (0, 0) if q is None else _head_rows(q, "q", dtype, B, T, dk)
    k_rows = (0, 0) if k is None else _head_rows(k, "k", dtype, B, T, dk)
    nm = _NORMS.get(norm)
    if nm is None:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}, got {norm!r}")
    if wq is not None:
        _check(wq, "wq", _F32, (dk,))
    if wk is not None:
        _check(wk, "wk", _F32, (dk,))
    rot = axes = 0
    if inv_freq is not None:
        _check(inv_freq, "inv_freq", _F32)
        pairs = inv_freq.numel()
        if inv_freq.dim() != 1 or 2 * pairs > dk:
            raise ValueError(f"inv_freq must be [rot/2] with rot <= {dk}, got {tuple(inv_freq.shape)}")
        rot, axes = 2 * pairs, 1
        if pos is not None:
            n = pos.dim()
            if n == 3:
                axes = pos.shape[0]
            if n not in (2, 3) or not 1 <= axes <= 4:
                raise ValueError(f"pos must be [B,T] or [axes,B,T] with 1 to 4 axes, got {tuple(pos.shape)}")
            _check(pos, "pos", torch.int32, (B, T) if n == 2 else (axes, B, T))
        if axis is not None:
            _check(axis, "axis", torch.int32, inv_freq.shape)
    elif pos is not None or axis is not None:
        raise ValueError("pos and axis need inv_freq")
    return B, T, dk, dt, nm, axes, rot, q_rows, k_rows


def qk_norm_rope_fwd(q, k, pos=None, inv_freq=None, wq=None, wk=None, norm="rms", eps=1e-6, axis=None,
                     interleaved=False, q_out=None, k_out=None, out_dtype=None, stream=None):
    """Queries and keys for the scans (see ``kdn_qk_norm_rope_fwd``): the norm
    of every head, the weight, the position rotation and the scans' layout.

    q [B,T,Hq,dk], k [B,T,Hk,dk] bf16 or fp32, dense or column slices of a
    fused projection (either may be None); ``pos`` [B,T] or [axes,B,T] int32
    (None: the token index); ``inv_freq`` [rot/2] fp32 (None: no rotation);
    ``wq``, ``wk`` [dk] fp32 or None; ``norm`` "rms", "l2" or "none"; ``axis``
    [rot/2] int32, the position axis of each pair, or None (the first);
    ``interleaved``: pairs (2p, 2p+1) instead of (p, p + rot/2).  Returns
    (q_out [B,Hq,T,dk], k_out [B,Hk,T,dk]) of ``out_dtype`` (q's by default)."""
    B, T, dk, it, nm, axes, rot, (Hq, q_ld), (Hk, k_ld) = _qk_common(q, k, pos, inv_freq, wq, wk, norm, axis)
    first = q if q is not None else k
    if q_out is not None and k_out is not None and q_out.dtype != k_out.dtype:
        raise ValueError("q_out and k_out must have one type")
    od = out_dtype or (q_out if q_out is not None else k_out if k_out is not None else first).dtype
    ot = _DTYPES.get(od)
    if ot is None:
        raise ValueError(f"the outputs must be bf16 or fp32, got {od}")
    if q is None:
        q_out = None
    elif q_out is None:
        q_out = _empty((B, Hq, T, dk), first, od, stream)
    else:
        _check(q_out, "q_out", od, (B, Hq, T, dk))
    if k is None:
        k_out = None
    elif k_out is None:
        k_out = _empty((B, Hk, T, dk), first, od, stream)
    else:
        _check(k_out, "k_out", od, (B, Hk, T, dk))
    if not _here(stream, q, k, pos, inv_freq, wq, wk, axis, q_out, k_out):
        _on_one_device(stream, q=q, k=k, pos=pos, inv_freq=inv_freq, wq=wq, wk=wk, axis=axis, q_out=q_out,
                       k_out=k_out)
    st = lib.kdn_qk_norm_rope_fwd(_ptr(q), q_ld, _ptr(k), k_ld, _ptr(wq), _ptr(wk), nm, eps, _ptr(pos),
                                  axes, _ptr(inv_freq), _ptr(axis), rot, int(interleaved), _ptr(q_out),
                                  _ptr(k_out), B, T, Hq, Hk, dk, it, ot, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_qk_norm_rope_fwd")
    return q_out, k_out


def qk_norm_rope_bwd_workspace(B, T, Hq, Hk, dk) -> int:
    """Bytes of device workspace ``qk_norm_rope_bwd`` needs."""
    _ints(B, T, Hq, Hk, dk)
    n = ctypes.c_longlong(0)
    st = lib.kdn_qk_norm_rope_bwd_workspace(B, T, Hq, Hk, dk, ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, "kdn_qk_norm_rope_bwd_workspace")
    return int(n.value)


@functools.lru_cache(maxsize=256)
def _qk_ws(device, B, T, Hq, Hk, dk):
    return qk_norm_rope_bwd_workspace(B, T, Hq, Hk, dk)


def qk_norm_rope_bwd(q, k, grad_q_out, grad_k_out, pos=None, inv_freq=None, wq=None, wk=None, norm="rms",
                     eps=1e-6, axis=None, interleaved=False, grad_q=None, grad_k=None, grad_w=None,
                     workspace=None, stream=None):
    """Backward pass of ``qk_norm_rope_fwd`` (see ``kdn_qk_norm_rope_bwd``):
    its inputs, and the gradients of its outputs ([B,H,T,dk], bf16 or fp32;
    ``diag_scan_bwd``'s q and k as they are).  ``grad_q``, ``grad_k``: tensors
    of q's type to write, dense or column slices of a fused gradient, or None
    (allocate).  ``grad_w``: whether the weights' gradients are wanted (None:
    of those given).  Returns a dict q, k [B,T,H,dk] and wq, wk [dk] fp32 or
    None."""
    B, T, dk, it, nm, axes, rot, (Hq, q_ld), (Hk, k_ld) = _qk_common(q, k, pos, inv_freq, wq, wk, norm, axis)
    first = q if q is not None else k
    g = {}
    lds = {}
    gts = []
    for name, t, H, go, gx, w in (("q", q, Hq, grad_q_out, grad_q, wq), ("k", k, Hk, grad_k_out, grad_k, wk)):
        g[name], lds[name], g["w" + name] = None, 0, None
        if t is None:
            continue
        if go is None:
            raise ValueError(f"grad_{name}_out must be given with {name}")
        _check(go, f"grad_{name}_out", None, (B, H, T, dk))
        gts.append(go.dtype)
        if gx is None:
            # (dense: t's heads lie side by side, so what empty_like makes of its order is the plain one)
            g[name] = (torch.empty_like(t, memory_format=torch.contiguous_format) if stream is None
                       else _dense_like(t, stream))
            lds[name] = H * dk
        else:
            g[name] = gx
            n, lds[name] = _head_rows(gx, "grad_" + name, t.dtype, B, T, dk)
            if n != H:
                raise ValueError(f"grad_{name} must have {H} heads, got {n}")
        if (w is not None) if grad_w is None else grad_w:
            if H == 0:                                         # (nothing writes it)
                with _alloc(stream):
                    g["w" + name] = torch.zeros(dk, device=t.device, dtype=_F32)
            else:
                g["w" + name] = (_empty(dk, t, _F32, stream) if w is None else
                                 torch.empty_like(w) if stream is None else _dense_like(w, stream))
    if len(set(gts)) > 1:
        raise ValueError("grad_q_out and grad_k_out must have one type")
    ot = _DTYPES.get(gts[0])
    if ot is None:
        raise ValueError(f"the outputs' gradients must be bf16 or fp32, got {gts[0]}")
    ws_bytes = 0
    if g["wq"] is not None or g["wk"] is not None:
        ws_bytes = _qk_ws(_ws_device(first), B, T, Hq, Hk, dk)
        if workspace is None:
            workspace = _scratch(ws_bytes, first, stream)
        else:
            _check_workspace(workspace, ws_bytes)
    else:
        workspace = None
    grad_q_out, grad_k_out = None if q is None else grad_q_out, None if k is None else grad_k_out
    if not _here(stream, q, k, grad_q_out, grad_k_out, pos, inv_freq, wq, wk, axis, g["q"], g["k"], workspace):
        _on_one_device(stream, q=q, k=k, grad_q_out=grad_q_out, grad_k_out=grad_k_out, pos=pos, inv_freq=inv_freq,
                       wq=wq, wk=wk, axis=axis, grad_q=g["q"], grad_k=g["k"], workspace=workspace)
    st = lib.kdn_qk_norm_rope_bwd(_ptr(q), q_ld, _ptr(k), k_ld, _ptr(wq), _ptr(wk), nm, float(eps), _ptr(pos),
                                  axes, _ptr(inv_freq), _ptr(axis), rot, int(interleaved),
                                  _ptr(grad_q_out), _ptr(grad_k_out), _ptr(g["q"]), lds["q"], _ptr(g["k"]),
                                  lds["k"], _ptr(g["wq"]), _ptr(g["wk"]), B, T, Hq, Hk, dk, it, ot,
                                  _ptr(workspace), ws_bytes, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_qk_norm_rope_bwd")
    return g


# ---------------------------------------------------------------------------
# the gated delta rule

def _delta_sizes(q, v, offsets):
    """(B, H, T, dk, dv, nseq, shape of the states) of a delta-rule call."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"q must be [B,H,T,dk] and v [B,H,T,dv], got {tuple(q.shape)} and {tuple(v.shape)}")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    rows, nseq = B, 0
    if offsets is not None:
        _check(offsets, "offsets", torch.int32)
        if offsets.dim() != 1 or offsets.numel() < 2 or B != 1:
            raise ValueError("offsets must be [nseq + 1] with B = 1")
        rows = nseq = offsets.numel() - 1
    if (B | H | T | dk | dv | rows) > _MOST:
        _ints(B, H, T, dk, dv, rows)
    return B, H, T, dk, dv, nseq, (rows, H, dv, dk)


def _delta_inputs(q, k, v, beta, d, A, S0, shape, state):
    """Checks what the forward and the backward share; returns in_dtype."""
    B, H, T, dk, dv = shape
    it, dt = _dtype_of(q, "q"), q.dtype
    _check(q, "q", dt)
    _check(k, "k", dt, q.shape)
    _check(v, "v", dt, (B, H, T, dv))
    _check(beta, "beta", dt, (B, H, T))
    _check(d, "d", dt, (B, H, T))
    _check(A, "A", _F32, (H,))
    if S0 is not None:
        _check(S0, "S0", _F32, state)
    return it


def _delta_workspace(f, what, B, H, T, dk, dv, nseq, dtype):
    _ints(B, H, T, dk, dv, nseq)
    n = ctypes.c_longlong(0)
    st = f(B, H, T, dk, dv, nseq, KDN_BF16 if dtype == torch.bfloat16 else KDN_F32, ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, what)
    return int(n.value)


def delta_scan_fwd_workspace(B, H, T, dk, dv, nseq=0, dtype=torch.bfloat16) -> int:
    """Bytes of device workspace ``delta_scan_fwd`` needs (0: none)."""
    return _delta_workspace(lib.kdn_delta_scan_fwd_workspace, "kdn_delta_scan_fwd_workspace", B, H, T, dk, dv, nseq,
                            dtype)


def delta_scan_bwd_workspace(B, H, T, dk, dv, nseq=0, dtype=torch.bfloat16) -> int:
    """Bytes of device workspace ``delta_scan_bwd`` needs."""
    return _delta_workspace(lib.kdn_delta_scan_bwd_workspace, "kdn_delta_scan_bwd_workspace", B, H, T, dk, dv, nseq,
                            dtype)


@functools.lru_cache(maxsize=512)
def _delta_ws(device, back, *sizes):
    return (delta_scan_bwd_workspace if back else delta_scan_fwd_workspace)(*sizes)


def delta_scan_fwd(q, k, v, beta, d, A, S0=None, offsets=None, out=None, out_dtype=None, final_state=True,
                   workspace=None, stream=None):
    """The gated delta rule S_t = alpha_t S_{t-1} + beta_t (v_t - alpha_t
    S_{t-1} k_t) k_t^T, o_t = S_t q_t, alpha_t = exp(-A d_t) (see
    ``kdn_delta_scan_fwd``).

    q, k [B,H,T,dk], v [B,H,T,dv], beta, d [B,H,T] (bf16 or fp32, all the
    same); A [H] fp32; S0 [B,H,dv,dk] fp32 or None.  ``offsets`` [nseq + 1]
    int32 (device): packed sequences with B = 1; S0 and final_state are then
    [nseq,H,dv,dk].  ``out_dtype`` is out's type (q's by default);
    ``final_state`` True (allocate), False/None (skip) or a tensor.
    ``workspace``: a uint8 device tensor of at least
    ``delta_scan_fwd_workspace`` bytes, or None (one is taken from torch's
    caching allocator for the call).  Returns (out [B,H,T,dv], final_state or
    None).  With offsets, tokens of an ``out`` allocated here that lie in no
    sequence are undefined."""
    B, H, T, dk, dv, nseq, state = _delta_sizes(q, v, offsets)
    it = _delta_inputs(q, k, v, beta, d, A, S0, (B, H, T, dk, dv), state)
    if out is None:
        out = _new(v, out_dtype, stream)
    else:
        _check(out, "out", out_dtype, v.shape)
    ot = _dtype_of(out, "out")
    if final_state is True:
        final_state = _empty(state, q, _F32, stream)
    elif final_state is False:
        final_state = None
    elif final_state is not None:
        _check(final_state, "final_state", _F32, state)
    ws_bytes = _delta_ws(_ws_device(q), False, B, H, T, dk, dv, nseq, q.dtype)
    if workspace is not None:
        _check_workspace(workspace, ws_bytes)
    elif ws_bytes:
        workspace = _scratch(ws_bytes, q, stream)
    if not _here(stream, q, k, v, beta, d, A, S0, offsets, out, final_state, workspace):
        _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, S0=S0, offsets=offsets, out=out,
                       final_state=final_state, workspace=workspace)
    st = lib.kdn_delta_scan_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A), _ptr(S0), _ptr(offsets),
                                nseq, _ptr(out), _ptr(final_state), B, H, T, dk, dv, it, ot, _ptr(workspace),
                                ws_bytes, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_delta_scan_fwd")
    return out, final_state


def delta_scan_bwd(q, k, v, beta, d, A, grad_out, S0=None, offsets=None, grad_final_state=None, grad_q=None,
                   grad_k=None, grad_v=None, grad_beta=None, grad_d=None, grad_A=True, grad_S0=True,
                   workspace=None, stream=None):
    """Backward pass of ``delta_scan_fwd`` (see ``kdn_delta_scan_bwd``): its
    inputs, and ``grad_out`` [B,H,T,dv] of out's type.  ``grad_q`` ...
    ``grad_d``: tensors of the inputs' type and shape to write, or None
    (allocate); ``grad_A``, ``grad_S0``: True (allocate), False/None (skip) or
    fp32 tensors.  Returns a dict q, k, v, beta, d, A, S0.  ``workspace``: a
    uint8 device tensor of at least ``delta_scan_bwd_workspace`` bytes, or
    None (one is taken from torch's caching allocator for the call).  With
    offsets, gradients allocated here are undefined for tokens that lie in no
    sequence."""
    B, H, T, dk, dv, nseq, state = _delta_sizes(q, v, offsets)
    it = _delta_inputs(q, k, v, beta, d, A, S0, (B, H, T, dk, dv), state)
    ot = _dtype_of(grad_out, "grad_out")
    _check(grad_out, "grad_out", None, v.shape)
    if grad_final_state is not None:
        _check(grad_final_state, "grad_final_state", _F32, state)
    g = {}
    for name, like, t in (("q", q, grad_q), ("k", k, grad_k), ("v", v, grad_v), ("beta", beta, grad_beta),
                          ("d", d, grad_d)):
        if t is None:
            t = _new(like, None, stream)
        else:
            _check(t, "grad_" + name, q.dtype, like.shape)
        g[name] = t
    for name, t, shape in (("A", grad_A, (H,)), ("S0", grad_S0, state)):
        if t is True:
            t = _empty(shape, q, _F32, stream)
        elif t is False:
            t = None
        elif t is not None:
            _check(t, "grad_" + name, _F32, shape)
        g[name] = t
    ws_bytes = _delta_ws(_ws_device(q), True, B, H, T, dk, dv, nseq, q.dtype)
    if workspace is not None:
        _check_workspace(workspace, ws_bytes)
    elif ws_bytes:
        workspace = _scratch(ws_bytes, q, stream)
    if not _here(stream, q, k, v, beta, d, A, S0, offsets, grad_out, grad_final_state, *g.values(), workspace):
        _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, S0=S0, offsets=offsets, grad_out=grad_out,
                       grad_final_state=grad_final_state, workspace=workspace,
                       **{"grad_" + n: t for n, t in g.items()})
    st = lib.kdn_delta_scan_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A), _ptr(S0), _ptr(offsets),
                                nseq, _ptr(grad_out), _ptr(grad_final_state), _ptr(g["q"]), _ptr(g["k"]),
                                _ptr(g["v"]), _ptr(g["beta"]), _ptr(g["d"]), _ptr(g["A"]), _ptr(g["S0"]), B, H, T,
                                dk, dv, it, ot, _ptr(workspace), ws_bytes, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_delta_scan_bwd")
    return g


def delta_step(q, k, v, beta, d, A, state, new_state=None, out=None, out_dtype=None, stream=None):
    """One token of ``delta_scan_fwd`` from a device-resident state (see
    ``kdn_delta_step``): q, k [B,H,dk]; v [B,H,dv]; beta, d [B,H] (bf16 or
    fp32, all the same); A [H] fp32; state [B,H,dv,dk] fp32, updated in place,
    or left as it is when ``new_state`` is another tensor to write.  Returns
    out [B,H,dv] (q's type unless ``out_dtype`` says otherwise)."""
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError(f"q must be [B,H,dk] and v [B,H,dv], got {tuple(q.shape)} and {tuple(v.shape)}")
    (B, H, dk), dv, dt = q.shape, v.shape[2], q.dtype
    if (B | H | dk | dv) > _MOST:
        _ints(B, H, dk, dv)
    it = _dtype_of(q, "q")
    if new_state is None:
        new_state = state
    if out is None:
        out = _new(v, out_dtype, stream)
    # a step is a few microseconds: one expression where all is well, the
    # messages where it is not
    heads, rows, states = (B, H), (B, H, dv), (B, H, dv, dk)
    if not (k.dtype is dt and v.dtype is dt and beta.dtype is dt and d.dtype is dt and A.dtype is _F32
            and state.dtype is _F32 and new_state.dtype is _F32 and (out_dtype is None or out.dtype is out_dtype)
            and k.shape == q.shape and v.shape == rows and out.shape == rows and beta.shape == heads
            and d.shape == heads and A.shape == (H,) and state.shape == states and new_state.shape == states
            and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and beta.is_contiguous()
            and d.is_contiguous() and A.is_contiguous() and state.is_contiguous() and new_state.is_contiguous()
            and out.is_contiguous()):
        for name, t, dtype, shape in (("q", q, dt, None), ("k", k, dt, q.shape), ("v", v, dt, rows),
                                      ("beta", beta, dt, heads), ("d", d, dt, heads), ("A", A, _F32, (H,)),
                                      ("state", state, _F32, states), ("new_state", new_state, _F32, states),
                                      ("out", out, out_dtype, rows)):
            _check(t, name, dtype, shape)
    ot = _dtype_of(out, "out")
    if not _here(stream, q, k, v, beta, d, A, state, new_state, out):
        _on_one_device(stream, q=q, k=k, v=v, beta=beta, d=d, A=A, state=state, new_state=new_state, out=out)
    st = lib.kdn_delta_step(q.data_ptr(), k.data_ptr(), v.data_ptr(), beta.data_ptr(), d.data_ptr(), A.data_ptr(),
                            state.data_ptr(), new_state.data_ptr(), out.data_ptr(), B, H, dk, dv, it, ot,
                            _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_delta_step")
    return out


# ---------------------------------------------------------------------------
# the residual's addition and its norm

_GROUP = 128                                                 # channels to a scale of an 8-bit output


def _rows_ld(t, name):
    """(rows, C, elements between rows) of a [..., C] tensor whose channels
    are adjacent and whose rows are evenly apart (dense, or a column slice of
    a wider tensor)."""
    shape = t.shape
    if len(shape) < 1 or shape[-1] < 1:
        raise ValueError(f"{name} must be [..., C] with C > 0, got {tuple(shape)}")
    C = shape[-1]
    rows = t.numel() // C
    if C > _MOST:
        _ints(C)
    if t.is_contiguous():
        return rows, C, C
    st, ld, step = t.stride(), None, None
    if C > 1 and st[-1] != 1:
        raise ValueError(f"{name} must have adjacent channels")
    for n, s in zip(reversed(t.shape[:-1]), reversed(st[:-1])):
        if n > 1:
            if ld is None:
                ld = step = s
            if s != step:
                raise ValueError(f"{name}'s rows must be evenly apart (stride {step}), got stride {s}")
            step *= n
    ld = C if ld is None else ld
    if ld < C:
        raise ValueError(f"{name}'s rows must be apart by at least their channels")
    return rows, C, ld


def add_rms_norm_fwd(x, residual=None, weight=None, eps=1e-6, sum_out=None, out=None, out_dtype=None, scale=None,
                     stream=None):
    """s = x + residual and y = weight . s / sqrt(mean(s^2) + eps) over the
    last dimension (see ``kdn_add_rms_norm_fwd``).

    x [...,C] bf16 or fp32, dense or a column slice; ``residual`` of x's shape,
    bf16 or fp32, or None; ``weight`` [C] fp32 or None.  ``sum_out``: a tensor
    of residual's type to write s to (residual itself: in place), or None
    (allocate).  ``out_dtype``: y's type (x's by default);
    ``torch.float8_e4m3fn`` gives y / scale in 8 bits with a ``scale``
    [...,ceil(C/128)] fp32, one for each 128 channels (allocated unless
    given).  Returns (y, s, scale): s is x where there is no residual, scale
    None where y is not in 8 bits."""
    rows, C, ld = _rows_ld(x, "x")
    xt = _dtype_of(x, "x")
    if residual is None:
        if sum_out is not None:
            raise ValueError("sum_out needs a residual")
        rt = xt
    else:
        rt = _dtype_of(residual, "residual")
        _check(residual, "residual", None, x.shape)
        if sum_out is None:
            sum_out = _new(residual, None, stream)
        else:
            _check(sum_out, "sum_out", residual.dtype, x.shape)
    if weight is not None:
        _check(weight, "weight", _F32, (C,))
    if out is None:
        out = _new(x, out_dtype, stream)
    else:
        _check(out, "out", out_dtype, x.shape)
    if out.dtype is torch.float8_e4m3fn:
        yt, shape = KDN_E4M3, (*x.shape[:-1], -(-C // _GROUP))
        if scale is None:
            scale = _empty(shape, x, _F32, stream)
        else:
            _check(scale, "scale", _F32, shape)
    else:
        yt = _DTYPES.get(out.dtype)
        if yt is None:
            raise ValueError(f"out must be bf16, fp32 or float8_e4m3fn, got {out.dtype}")
        if scale is not None:
            raise ValueError("scale needs an output in 8 bits")
    if not _here(stream, x, residual, weight, sum_out, out, scale):
        _on_one_device(stream, x=x, residual=residual, weight=weight, sum_out=sum_out, out=out, scale=scale)
    st = lib.kdn_add_rms_norm_fwd(x.data_ptr(), ld, _ptr(residual), _ptr(weight), eps, _ptr(sum_out), out.data_ptr(),
                                  _ptr(scale), rows, C, xt, rt, yt, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_add_rms_norm_fwd")
    return out, x if residual is None else sum_out, scale


def add_rms_norm_bwd_workspace(rows, C) -> int:
    """Bytes of device workspace ``add_rms_norm_bwd`` needs."""
    _ints(rows, C)
    n = ctypes.c_longlong(0)
    st = lib.kdn_add_rms_norm_bwd_workspace(rows, C, ctypes.byref(n))
    if st != KDN_OK:
        raise KdnError(st, "kdn_add_rms_norm_bwd_workspace")
    return int(n.value)


@functools.lru_cache(maxsize=256)
def _norm_ws(device, rows, C):
    return add_rms_norm_bwd_workspace(rows, C)


def add_rms_norm_bwd(sum, grad_y, weight=None, grad_sum=None, eps=1e-6, x_dtype=None, grad_residual=None, grad_x=None,
                     grad_weight=None, workspace=None, stream=None):
    """Backward pass of ``add_rms_norm_fwd`` with y in bf16 or fp32 (see
    ``kdn_add_rms_norm_bwd``): ``sum`` [...,C] is the s that it returned (a
    column slice is copied to dense rows first), ``grad_y`` of y's type,
    ``grad_sum`` the gradient that comes to s from further on (sum's type) or
    None.  ``grad_residual``: a tensor of sum's type to write (grad_sum itself:
    in place) or None (allocate); ``grad_x`` the same in ``x_dtype`` (sum's by
    default: then one tensor serves both, unless grad_x is given).
    ``grad_weight``: whether the weight's gradient is wanted (None: of one
    given).  Returns a dict residual, x [...,C] and weight [C] fp32 or None."""
    rows, C, _ = _rows_ld(sum, "sum")
    if not sum.is_contiguous():                              # the forward's x as it was; the kernel reads dense rows
        with _alloc(stream):
            sum = sum.contiguous()
    rt = _dtype_of(sum, "sum")
    yt = _dtype_of(grad_y, "grad_y")
    _check(grad_y, "grad_y", None, sum.shape)
    if weight is not None:
        _check(weight, "weight", _F32, (C,))
    if grad_sum is not None:
        _check(grad_sum, "grad_sum", sum.dtype, sum.shape)
    if grad_residual is None:
        grad_residual = _new(sum, None, stream)
    else:
        _check(grad_residual, "grad_residual", sum.dtype, sum.shape)
    if grad_x is not None:
        _check(grad_x, "grad_x", x_dtype, sum.shape)
    elif x_dtype is not None and x_dtype is not sum.dtype:
        grad_x = _empty(sum.shape, sum, x_dtype, stream)
    xt = rt if grad_x is None else _dtype_of(grad_x, "grad_x")
    gw, ws_bytes = None, 0
    if (weight is not None) if grad_weight is None else grad_weight:
        gw = _empty(C, sum, _F32, stream)
        ws_bytes = _norm_ws(_ws_device(sum), rows, C)
        if workspace is None:
            workspace = _scratch(ws_bytes, sum, stream)
        else:
            _check_workspace(workspace, ws_bytes)
    else:
        workspace = None
    if not _here(stream, sum, grad_y, weight, grad_sum, grad_residual, grad_x, gw, workspace):
        _on_one_device(stream, sum=sum, grad_y=grad_y, weight=weight, grad_sum=grad_sum,
                       grad_residual=grad_residual, grad_x=grad_x, grad_weight=gw, workspace=workspace)
    st = lib.kdn_add_rms_norm_bwd(sum.data_ptr(), _ptr(weight), eps, grad_y.data_ptr(), _ptr(grad_sum),
                                  grad_residual.data_ptr(), _ptr(grad_x), _ptr(gw), rows, C, xt, rt, yt,
                                  _ptr(workspace), ws_bytes, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_add_rms_norm_bwd")
    return dict(residual=grad_residual, x=grad_residual if grad_x is None else grad_x, weight=gw)


def diag_scan_plan(B, H, T, dk, dv, dtype=torch.bfloat16) -> dict:
    """Launch plan of a diagonal-scan call: token parts, kernels, scratch bytes."""
    p, k, sb = ctypes.c_int(), ctypes.c_int(), ctypes.c_longlong()
    st = lib.kdn_diag_scan_plan(B, H, T, dk, dv, KDN_BF16 if dtype == torch.bfloat16 else KDN_F32,
                                ctypes.byref(p), ctypes.byref(k), ctypes.byref(sb))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_scan_plan")
    return dict(parts=p.value, kernels=k.value, scratch_bytes=sb.value)


def mobius_scan_plan(N, T) -> dict:
    """Launch plan of a Moebius-scan call: kernels and scratch bytes."""
    k, sb = ctypes.c_int(), ctypes.c_longlong()
    st = lib.kdn_mobius_scan_plan(N, T, ctypes.byref(k), ctypes.byref(sb))
    if st != KDN_OK:
        raise KdnError(st, "kdn_mobius_scan_plan")
    return dict(kernels=k.value, scratch_bytes=sb.value)


MOBIUS_NOALLOC_MAX_TILES = 43690   # N * ceil(T / 2048) limit of mobius_scan_noalloc


def mobius_scan_noalloc(a, b, c, d, lambda0, out, stream=None):
    """``kdn_mobius_scan_noalloc``: the Moebius scan for callers that must not
    allocate device memory during the call (e.g. a framework that reserved
    the GPU's memory up front).  The caller passes every buffer, ``out``
    included; the look-back scratch is a fixed 1 MiB array in the library.
    Calls that overlap on the GPU share that array and race."""
    N, T = a.shape
    for name, t in (("a", a), ("b", b), ("c", c), ("d", d), ("out", out)):
        _check(t, name, torch.float32, (N, T))
    _check(lambda0, "lambda0", torch.float32, (N,))
    _on_one_device(stream, a=a, b=b, c=c, d=d, lambda0=lambda0, out=out)
    st = lib.kdn_mobius_scan_noalloc(_ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(lambda0), _ptr(out),
                                     N, T, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_mobius_scan_noalloc")
    return out


def get_device_error(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device error word."""
    return int(lib.kdn_get_device_error(_stream(stream)))


def set_wait_limit_ns(ns: int) -> None:
    lib.kdn_set_wait_limit_ns(int(ns))


def debug_stall_mobius_tile(tile: int) -> None:
    lib.kdn_debug_stall_mobius_tile(int(tile))


def debug_stall_gated_rank(rank: int) -> None:
    lib.kdn_debug_stall_gated_rank(int(rank))


def debug_stall_delta_chunk(chunk: int) -> None:
    lib.kdn_debug_stall_delta_chunk(int(chunk))


# ---------------------------------------------------------------------------
# host-buffer calls: kdn_diag_scan_fwd_host / kdn_mobius_scan_host copy in,
# scan and copy out in pipelined chunks (page-locked tensors let the copies
# overlap the scans); results land in host tensors.

def _host_out(t, name, shape):
    """A caller-given host output (checked) or a new page-locked one."""
    if t is None:
        return torch.empty(shape, dtype=torch.float32, pin_memory=True)
    if t.is_cuda:
        raise ValueError(f"{name} must be a host tensor when the inputs are")
    _check(t, name, torch.float32, shape)
    return t


def _diag_host(q, k, v, beta, d, A, I_prior, I0, mu0, out, final_state, stream):
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    if dt not in (torch.bfloat16, torch.float32):
        raise ValueError("inputs must be bf16 or fp32")
    for name, t, shape, dtype in (("q", q, (B, H, T, dk), dt), ("k", k, (B, H, T, dk), dt),
                                  ("v", v, (B, H, T, dv), dt), ("beta", beta, (B, H, T, dv), dt),
                                  ("d", d, (B, H, T), dt), ("A", A, (H,), torch.float32),
                                  ("I0", I0, (B, H, dv, dk), torch.float32),
                                  ("mu0", mu0, (B, H, dv, dk), torch.float32)):
        if t is not None:
            if t.is_cuda:
                raise ValueError(f"{name} must be a host tensor like q")
            _check(t, name, dtype, shape)
    out = _host_out(out, "out", (B, H, T, dv))
    if final_state is True:
        final_state = None
        fs = _host_out(None, "final_state", (2, B, H, dv, dk))
    elif final_state is False or final_state is None:
        fs = None
    else:
        fs = _host_out(final_state, "final_state", (2, B, H, dv, dk))
    st = lib.kdn_diag_scan_fwd_host(_ptr(q), _ptr(k), _ptr(v), _ptr(beta), _ptr(d), _ptr(A),
                                    float(I_prior), _ptr(I0), _ptr(mu0), _ptr(out), _ptr(fs),
                                    B, H, T, dk, dv, KDN_BF16 if dt == torch.bfloat16 else KDN_F32,
                                    _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_diag_scan_fwd_host")
    return out, fs


def _mobius_host(a, b, c, d, lambda0, out, stream):
    N, T = a.shape
    for name, t in (("a", a), ("b", b), ("c", c), ("d", d)):
        if t.is_cuda:
            raise ValueError(f"{name} must be a host tensor like a")
        _check(t, name, torch.float32, (N, T))
    _check(lambda0, "lambda0", torch.float32, (N,))
    out = _host_out(out, "out", (N, T))
    st = lib.kdn_mobius_scan_host(_ptr(a), _ptr(b), _ptr(c), _ptr(d), _ptr(lambda0), _ptr(out),
                                  N, T, _stream(stream))
    if st != KDN_OK:
        raise KdnError(st, "kdn_mobius_scan_host")
    return out
