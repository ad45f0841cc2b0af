"""The residual update with its norm, and gradient clipping (include/ssm_train.h).

Output tensors that a caller gives overlap no input and no other output,
except where a function says so.
"""
from __future__ import annotations

import ctypes

import torch

from . import SsmError, lib
from . import _check
from .linattn import _IO, _bad, _current_device, _dense, _gpu, _on, _raw_stream, _workspace

_VP, _I64 = ctypes.c_void_p, ctypes.c_int64
lib.ssm_add_norm.argtypes = [_I64, _I64, ctypes.c_int32, _VP, _VP, _VP, ctypes.c_float, _VP, _VP, _VP, _VP]
lib.ssm_add_norm.restype = ctypes.c_int
lib.ssm_add_norm_grad_workspace_bytes.argtypes = [_I64, _I64]
lib.ssm_add_norm_grad_workspace_bytes.restype = ctypes.c_size_t
lib.ssm_add_norm_grad.argtypes = [_I64, _I64, ctypes.c_int32] + [_VP] * 8 + [ctypes.c_size_t, _VP]
lib.ssm_add_norm_grad.restype = ctypes.c_int
lib.ssm_clip_grads_workspace_bytes.argtypes = [ctypes.c_int32, ctypes.POINTER(_I64)]
lib.ssm_clip_grads_workspace_bytes.restype = ctypes.c_size_t
lib.ssm_clip_grads.argtypes = [ctypes.c_int32, ctypes.POINTER(_VP), ctypes.POINTER(_VP), ctypes.POINTER(_I64),
                               ctypes.c_int32, ctypes.c_float, _VP, _VP, ctypes.c_size_t, _VP]
lib.ssm_clip_grads.restype = ctypes.c_int

_F32 = torch.float32


def _sizes(t, name: str):
    """Rows and channels of a float32 tensor [..., P]."""
    shape = t.shape
    if len(shape) < 2 or t.numel() == 0:
        _bad(f"{name}: expected rows of channels, got shape {tuple(shape)}")
    return t.numel() // shape[-1], shape[-1]


def add_norm(r, y, norm_scale, eps=1e-5, r_out=None, x=None, rinv=None, io=None, stream=None):
    """r_out = r + y and x = norm_scale r_out / rms(r_out); returns (x, r_out,
    rinv).  r [..., P] float32; y of the same shape in the io dtype, or None
    (then r_out is r itself unless given, and io, "f32" or "bf16", names x's
    dtype).  r_out may be r.  rinv [...] float32 is 1 / rms, for the gradient."""
    device = _gpu(r, "r", None, _F32)
    if stream is not None or device != _current_device():
        with _on(device, stream):
            return add_norm(r, y, norm_scale, eps, r_out, x, rinv, io)
    T, P = _sizes(r, "r")
    shape = r.shape
    like = y if y is not None else x
    if like is not None:
        _gpu(like, "y" if y is not None else "x", device)
        dt = like.dtype
    else:
        dt = {"f32": _F32, "bf16": torch.bfloat16}.get(io)
    if dt not in _IO:
        _bad("the io dtype is bfloat16 or float32")
    if norm_scale is None:
        _bad("norm_scale is required")
    rp = _dense(r, "r", shape, device, _F32)
    yp = _dense(y, "y", shape, device, dt)
    gp = _dense(norm_scale, "norm_scale", (P,), device, _F32)
    if r_out is None:
        r_out = r if y is None else torch.empty_like(r)
    elif r_out is not r:
        _dense(r_out, "r_out", shape, device, _F32)
    if x is None:
        x = torch.empty_like(r if y is None else y, dtype=dt)
    else:
        _dense(x, "x", shape, device, dt)
    if rinv is None:
        rinv = r.new_empty(T if len(shape) == 2 else shape[:-1])
    else:
        _dense(rinv, "rinv", shape[:-1], device, _F32)
    _check(lib.ssm_add_norm(T, P, _IO[dt], rp, yp, gp, eps, r_out.data_ptr(), x.data_ptr(), rinv.data_ptr(),
                            _raw_stream(device)), "ssm_add_norm")
    return x, r_out, rinv


def add_norm_grad(r_out, rinv, norm_scale, dx, dr_out=None, dr=None, want_scale=True, ws=None, stream=None):
    """Gradient of add_norm; returns (dr, dnorm_scale).  dr (float32) is the
    cotangent of r and of y: dr_out, the cotangent of r_out from elsewhere
    (None: zero), plus the norm's part.  dr may be dr_out."""
    device = _gpu(r_out, "r_out", None, _F32)
    if stream is not None or device != _current_device():
        with _on(device, stream):
            return add_norm_grad(r_out, rinv, norm_scale, dx, dr_out, dr, want_scale, ws)
    T, P = _sizes(r_out, "r_out")
    shape = r_out.shape
    _gpu(dx, "dx", device)
    dt = dx.dtype
    if dt not in _IO:
        _bad(f"dx: dtype {dt}, expected bfloat16 or float32")
    if rinv is None or norm_scale is None:
        _bad("rinv and norm_scale are required")
    rp = _dense(r_out, "r_out", shape, device, _F32)
    ip = _dense(rinv, "rinv", shape[:-1], device, _F32)
    gp = _dense(norm_scale, "norm_scale", (P,), device, _F32)
    xp = _dense(dx, "dx", shape, device, dt)
    cp = _dense(dr_out, "dr_out", shape, device, _F32)
    nbytes = lib.ssm_add_norm_grad_workspace_bytes(T, P)
    if nbytes == 0:
        raise SsmError(4, "ssm_add_norm_grad_workspace_bytes")
    if dr is None:
        dr = torch.empty_like(r_out)
    dscale = torch.empty_like(norm_scale) if want_scale else None
    w = _workspace(ws, nbytes, device)
    _check(lib.ssm_add_norm_grad(T, P, _IO[dt], rp, ip, gp, xp, cp, _dense(dr, "dr", shape, device, _F32),
                                 None if dscale is None else dscale.data_ptr(), w.data_ptr(), w.numel(),
                                 _raw_stream(device)), "ssm_add_norm_grad")
    return dr, dscale


def _addresses(ts, name: str, device, dtype):
    """The addresses of contiguous tensors of one dtype on one device."""
    try:
        if all([t.get_device() == device and t.dtype is dtype and t.is_contiguous() for t in ts]):
            return [t.data_ptr() for t in ts]
    except AttributeError:
        pass  # not a tensor: refused below
    for t in ts:
        _gpu(t, name, device, dtype)
        if not t.is_contiguous():
            _bad(f"{name}: must be contiguous")


def _check_outputs(pi, po, ts):
    """Refuses an output given twice or that is another gradient (empty tensors share the null address)."""
    full = [i for i, t in enumerate(ts) if t.numel()]
    source = {pi[i]: i for i in full}
    if len({po[i] for i in full}) != len(full):
        _bad("clip_grads: an output is given twice")
    for i in full:
        if source.get(po[i], i) != i:
            _bad("clip_grads: an output is another gradient")


def clip_grads(grads, max_norm, out=None, norm=None, ws=None, stream=None):
    """Scales gradients to a global norm of at most max_norm; returns the norm
    before that, a float32 tensor [1] on the GPU (nothing is synchronised).
    grads: tensors, or dicts of tensors as adjoint_grad, stack_grad and
    linattn_grad return them, all of one dtype (float32 or bfloat16) on one
    GPU.  They are scaled in place, or into the tensors `out`, each of which may
    be its own gradient; a norm that is not finite leaves them as they are.  max_norm = inf only measures."""
    ts = []
    for g in grads:
        if isinstance(g, dict):
            ts.extend(t for t in g.values() if t is not None)
        else:
            ts.append(g)
    if not ts:
        _bad("clip_grads: no gradients")
    device = _gpu(ts[0], "grads[0]")
    if stream is not None or device != _current_device():
        with _on(device, stream):
            return clip_grads(ts, max_norm, out, norm, ws)
    dt = ts[0].dtype
    if dt not in _IO:
        _bad(f"grads: dtype {dt}, expected bfloat16 or float32")
    if not max_norm > 0:
        _bad("max_norm must be positive")
    n = len(ts)
    pi = _addresses(ts, "a gradient", device, dt)
    if out is None:
        po = pi
        if len(set(pi)) != n:
            used = [p for p, t in zip(pi, ts) if t.numel()]  # empty tensors share the null address
            if len(set(used)) != len(used):
                _bad("clip_grads: a gradient is given twice")
    else:
        out = list(out)
        if len(out) != n:
            _bad(f"clip_grads: {len(out)} outputs for {n} gradients")
        po = _addresses(out, "an output", device, dt)
        for o, t in zip(out, ts):
            if o.shape != t.shape:
                _bad(f"an output: shape {tuple(o.shape)}, expected {tuple(t.shape)}")
        used = set(po)
        if len(used) != n or not used.isdisjoint(pi):
            _check_outputs(pi, po, ts)
    ptrs, counts = _VP * n, _I64 * n
    ns = counts(*[t.numel() for t in ts])
    nbytes = lib.ssm_clip_grads_workspace_bytes(n, ns)
    if nbytes == 0:
        raise SsmError(4, "ssm_clip_grads_workspace_bytes")
    if norm is None:
        norm = torch.empty(1, dtype=_F32, device=ts[0].device)
    w = _workspace(ws, nbytes, device)
    measure = out is None and max_norm == float("inf")
    _check(lib.ssm_clip_grads(n, ptrs(*pi), None if measure else ptrs(*po), ns, _IO[dt], max_norm,
                              _dense(norm, "norm", (1,), device, _F32), w.data_ptr(), w.numel(), _raw_stream(device)),
           "ssm_clip_grads")
    return norm
