"""Linear attention with a decay for each head (include/ssm_linattn.h).

    h_t = e^{g_t} h_{t-1} + k_t v_t^T,   y_t = scale q_t^T h_t    per head

linattn_forward runs prompts or training sequences, linattn_grad their
gradient, linattn_step one token for each of a batch of sequences.  Tokens are
rows of q, k [T, Hk, dk] and v [T, Hv, dv] (Hk divides Hv; value head h reads
key head h // (Hv // Hk)); rows may be strided, heads and channels not.
Sequences are packed (seq_start, offsets on the GPU), or equally long when the
tensors are [S, L, H, d].  log_decay is float32, [T, Hv] or, one for each head,
[Hv]; states are float32 [S, Hv, dk, dv].

Every tensor of a call lives on one GPU; work goes to that GPU's current
stream, or to the raw handle `stream`, on which tensors that the call makes
are then allocated too.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import SSM_BF16, SSM_F32, SsmError, alloc_workspace, lib
from . import _check

_P, _VP = ctypes.POINTER, ctypes.c_void_p
_IO = {torch.bfloat16: SSM_BF16, torch.float32: SSM_F32}


class LinattnDims(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int64), ("S", ctypes.c_int32), ("Hk", ctypes.c_int32), ("Hv", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("io", ctypes.c_int32),
                ("decay_tokens", ctypes.c_int32), ("scale", ctypes.c_float)]


class LinattnIn(ctypes.Structure):
    _fields_ = [("q", _VP), ("k", _VP), ("v", _VP), ("ldq", ctypes.c_int64), ("ldk", ctypes.c_int64),
                ("ldv", ctypes.c_int64), ("log_decay", _VP), ("seq_start", _VP), ("h0", _VP)]


class LinattnGrads(ctypes.Structure):
    _fields_ = [("dq", _VP), ("dk", _VP), ("dv", _VP), ("dlog_decay", _VP), ("dh0", _VP)]


lib.ssm_linattn_workspace_bytes.argtypes = [_P(LinattnDims), _P(LinattnGrads), _P(ctypes.c_size_t)]
lib.ssm_linattn_forward.argtypes = [_P(LinattnDims), _P(LinattnIn), _VP, ctypes.c_int64, _VP, _VP, ctypes.c_size_t, _VP]
lib.ssm_linattn_grad.argtypes = [_P(LinattnDims), _P(LinattnIn), _VP, ctypes.c_int64, _VP, _P(LinattnGrads), _VP,
                                 ctypes.c_size_t, _VP]
lib.ssm_linattn_step.argtypes = [_P(LinattnDims), _P(LinattnIn), _VP, _VP, ctypes.c_int64, _VP]
for _f in (lib.ssm_linattn_workspace_bytes, lib.ssm_linattn_forward, lib.ssm_linattn_grad, lib.ssm_linattn_step):
    _f.restype = ctypes.c_int

GRADS = ("dq", "dk", "dv", "dlog_decay", "dh0")


def _bad(msg: str):
    raise SsmError(1, msg)


@contextlib.contextmanager
def _foreign(device, stream):
    """The given stream, or another device's current one, for the duration of a call."""
    if stream is not None:
        with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=device)):
            yield int(stream)
    else:
        with torch.cuda.device(device):
            yield torch.cuda.current_stream(device).cuda_stream


def _context(device, stream):
    if stream is None and device.index == torch.cuda.current_device():
        return contextlib.nullcontext(torch.cuda.current_stream(device).cuda_stream)
    return _foreign(device, stream)


def _gpu(t, name: str, device=None, dtype=None):
    if not isinstance(t, torch.Tensor):
        _bad(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if not t.is_cuda:
        _bad(f"{name}: must be a GPU tensor (got {t.device})")
    if device is not None and t.device != device:
        _bad(f"{name}: on {t.device}, the other tensors on {device}")
    if dtype is not None and t.dtype != dtype:
        _bad(f"{name}: dtype {t.dtype}, expected {dtype}")


def _dense(t, name: str, shape, device, dtype):
    """A contiguous tensor of this shape, or None."""
    if t is None:
        return None
    _gpu(t, name, device, dtype)
    if tuple(t.shape) != tuple(shape):
        _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        _bad(f"{name}: must be contiguous")
    return t.data_ptr()


def _rows(t, name: str, lead, device, dtype, H=None, d=None):
    """Token rows [*lead, H, d] with contiguous heads and channels: (H, d, elements between rows)."""
    _gpu(t, name, device, dtype)
    shape = t.shape
    n = len(lead)
    if len(shape) != n + 2 or tuple(shape[:n]) != tuple(lead):
        _bad(f"{name}: shape {tuple(shape)}, expected {tuple(lead)} rows of heads and channels")
    h, c = shape[n], shape[n + 1]
    if (H is not None and h != H) or (d is not None and c != d):
        _bad(f"{name}: {h} heads of {c} channels, expected {H} of {d}")
    if h < 1 or c < 1:
        _bad(f"{name}: empty heads")
    st = t.stride()
    if (c > 1 and st[n + 1] != 1) or (h > 1 and st[n] != c):
        _bad(f"{name}: heads and channels must be contiguous (strides {st})")
    rows = shape[n - 1]
    ld = st[n - 1] if rows > 1 else st[0] if n == 2 and shape[0] > 1 else h * c
    if n == 2 and shape[0] > 1 and st[0] != rows * ld:
        _bad(f"{name}: sequences must follow one another (strides {st})")
    return h, c, ld


def _setup(q, k, v, log_decay, scale, seq_start, step=False):
    """Checks the inputs; returns (dims, device, leading shape, LinattnIn)."""
    _gpu(q, "q")
    device, io = q.device, q.dtype
    if io not in _IO:
        _bad(f"q: dtype {io}, expected bfloat16 or float32")
    if q.dim() not in ((3,) if step else (3, 4)):
        _bad(f"q: {q.dim()} dimensions")
    lead = tuple(q.shape[:-2])
    Hk, dk, ldq = _rows(q, "q", lead, device, io)
    _, _, ldk = _rows(k, "k", lead, device, io, Hk, dk)
    Hv, dv, ldv = _rows(v, "v", lead, device, io)
    T = 1
    for n in lead:
        T *= n
    if T < 1:
        _bad("no tokens")
    S, starts = (lead[0] if len(lead) == 2 else 1), None
    if seq_start is not None:
        if len(lead) != 1:
            _bad("seq_start goes with packed tokens [T, H, d]")
        S = seq_start.numel() - 1 if isinstance(seq_start, torch.Tensor) else 0
        if S < 1:
            _bad("seq_start: an int32 tensor of at least two offsets")
        starts = _dense(seq_start, "seq_start", (S + 1,), device, torch.int32)
    _gpu(log_decay, "log_decay", device, torch.float32)
    tokens = log_decay.dim() != 1
    _dense(log_decay, "log_decay", lead + (Hv,) if tokens else (Hv,), device, torch.float32)
    dims = LinattnDims(T, S, Hk, Hv, dk, dv, _IO[io], 1 if tokens else 0, float(scale))
    ins = LinattnIn(q.data_ptr(), k.data_ptr(), v.data_ptr(), ldq, ldk, ldv, log_decay.data_ptr(), starts, None)
    return dims, device, lead, ins


def linattn_workspace_bytes(dims: LinattnDims, grads: LinattnGrads | None = None) -> int:
    """Workspace of linattn_forward, or of linattn_grad for the outputs set in grads."""
    n = ctypes.c_size_t(0)
    _check(lib.ssm_linattn_workspace_bytes(ctypes.byref(dims), None if grads is None else ctypes.byref(grads),
                                           ctypes.byref(n)), "ssm_linattn_workspace_bytes")
    return n.value


def _workspace(ws, nbytes: int, device):
    if ws is None:
        return alloc_workspace(nbytes, device) if nbytes else None
    _gpu(ws, "workspace", device, torch.uint8)
    if not ws.is_contiguous() or ws.numel() < nbytes:
        raise SsmError(2, f"workspace: {nbytes} contiguous bytes needed")
    return ws


def linattn_forward(q, k, v, log_decay, seq_start=None, h0=None, scale=1.0, want_state=False, y=None, hT=None,
                    ws=None, stream=None):
    """Runs ssm_linattn_forward; returns (y, hT), hT None unless want_state or
    given.  y has v's shape; hT may be h0.  With seq_start, rows of y outside
    the sequences are not written."""
    dims, device, lead, ins = _setup(q, k, v, log_decay, scale, seq_start)
    states = (dims.S, dims.Hv, dims.dk, dims.dv)
    ins.h0 = _dense(h0, "h0", states, device, torch.float32)
    with _context(device, stream) as handle:
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=device)
        _, _, ldy = _rows(y, "y", lead, device, q.dtype, dims.Hv, dims.dv)
        if hT is None and want_state:
            hT = torch.empty(states, dtype=torch.float32, device=device)
        end = _dense(hT, "hT", states, device, torch.float32)
        w = _workspace(ws, linattn_workspace_bytes(dims), device)
        _check(lib.ssm_linattn_forward(ctypes.byref(dims), ctypes.byref(ins), y.data_ptr(), ldy, end,
                                       None if w is None else w.data_ptr(), 0 if w is None else w.numel(), handle),
               "ssm_linattn_forward")
    return y, hT


def linattn_grad(q, k, v, log_decay, dy, seq_start=None, h0=None, dhT=None, scale=1.0, want=None, grads=None, ws=None,
                 stream=None) -> dict:
    """Runs ssm_linattn_grad; returns the gradient dict.  want: names among
    GRADS (default: all, dh0 only with an h0).  grads: output tensors by
    name (then they alone are computed)."""
    dims, device, lead, ins = _setup(q, k, v, log_decay, scale, seq_start)
    states = (dims.S, dims.Hv, dims.dk, dims.dv)
    ins.h0 = _dense(h0, "h0", states, device, torch.float32)
    end = _dense(dhT, "dhT", states, device, torch.float32)
    _, _, lddy = _rows(dy, "dy", lead, device, q.dtype, dims.Hv, dims.dv)
    like = {"dq": (q.shape, q.dtype), "dk": (k.shape, q.dtype), "dv": (v.shape, q.dtype),
            "dlog_decay": (log_decay.shape, torch.float32), "dh0": (states, torch.float32)}
    with _context(device, stream) as handle:
        if grads is None:
            names = want if want is not None else GRADS if h0 is not None else GRADS[:4]
            for n in names:
                if n not in like:
                    _bad(f"want: {n!r} is none of {GRADS}")
            grads = {n: torch.empty(like[n][0], dtype=like[n][1], device=device) for n in names}
        for n in grads:
            if n not in like:
                _bad(f"grads: {n!r} is none of {GRADS}")
        g = LinattnGrads(*(_dense(grads.get(n), n, like[n][0], device, like[n][1]) for n in GRADS))
        w = _workspace(ws, linattn_workspace_bytes(dims, g), device)
        _check(lib.ssm_linattn_grad(ctypes.byref(dims), ctypes.byref(ins), dy.data_ptr(), lddy, end, ctypes.byref(g),
                                    None if w is None else w.data_ptr(), 0 if w is None else w.numel(), handle),
               "ssm_linattn_grad")
    return grads


def linattn_step(q, k, v, log_decay, state, scale=1.0, y=None, stream=None):
    """Runs ssm_linattn_step: row t of q, k [B, Hk, dk] and v [B, Hv, dv] is
    the next token of the sequence with state[t] ([B, Hv, dk, dv], updated in
    place).  Returns y [B, Hv, dv]."""
    dims, device, lead, ins = _setup(q, k, v, log_decay, scale, None, step=True)
    if state is None:
        _bad("state is required")
    st = _dense(state, "state", (dims.T, dims.Hv, dims.dk, dims.dv), device, torch.float32)
    with _context(device, stream) as handle:
        if y is None:
            y = torch.empty(v.shape, dtype=v.dtype, device=device)
        _, _, ldy = _rows(y, "y", lead, device, q.dtype, dims.Hv, dims.dv)
        _check(lib.ssm_linattn_step(ctypes.byref(dims), ctypes.byref(ins), st, y.data_ptr(), ldy, handle),
               "ssm_linattn_step")
    return y
