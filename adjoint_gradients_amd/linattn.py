"""Linear attention with a decay for each head (include/ssm_linattn.h).

    h_t = e^{g_t} h_{t-1} + k_t v_t^T,   y_t = scale q_t^T h_t    per head

linattn_forward runs prompts or training sequences, linattn_grad their
gradient, linattn_step one token for each of a batch of sequences.  Tokens are
rows of q, k [T, Hk, dk] and v [T, Hv, dv] (Hk divides Hv; value head h reads
key head h // (Hv // Hk)); rows may be strided, heads and channels not.
Sequences are packed (seq_start, offsets on the GPU), or equally long when the
tensors are [S, L, H, d].  log_decay is float32, [T, Hv] or, one for each head,
[Hv]; states are float32 [S, Hv, dk, dv].  Output tensors that a caller gives
overlap no input and no other output, except hT, which may be h0.

Every tensor of a call lives on one GPU; work goes to that GPU's current
stream, or to the raw handle `stream`, on which tensors that the call makes
are then allocated too.
"""
from __future__ import annotations

import contextlib
import ctypes

import torch

from . import SSM_BF16, SSM_F32, SsmError, lib
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


_raw_stream = torch._C._cuda_getCurrentRawStream
_current_device = torch._C._cuda_getDevice


def _bad(msg: str):
    raise SsmError(1, msg)


@contextlib.contextmanager
def _on(device, stream):
    """Makes a tensor's device, and the raw stream handle if given, current."""
    if stream is None:
        with torch.cuda.device(device):
            yield
    else:
        with torch.cuda.stream(torch.cuda.ExternalStream(int(stream), device=device)):
            yield


def _gpu(t, name: str, device=None, dtype=None):
    """Refuses anything but a GPU tensor (of this device index and dtype); returns its device index."""
    if not isinstance(t, torch.Tensor):
        _bad(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    d = t.get_device()
    if d < 0:
        _bad(f"{name}: must be a GPU tensor (got {t.device})")
    if device is not None and d != device:
        _bad(f"{name}: on {t.device}, other tensors of the call on cuda:{device}")
    if dtype is not None and t.dtype is not dtype:
        _bad(f"{name}: dtype {t.dtype}, expected {dtype}")
    return d


def _dense(t, name: str, shape, device, dtype):
    """The address of a contiguous tensor of this shape; None for None."""
    if t is None:
        return None
    _gpu(t, name, device, dtype)
    if t.shape != shape:
        _bad(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        _bad(f"{name}: must be contiguous")
    return t.data_ptr()


def _rows(t, name: str, lead, device, dtype, heads=None):
    """Token rows [*lead, H, d] with contiguous heads and channels: ((H, d), elements between rows)."""
    _gpu(t, name, device, dtype)
    shape = t.shape
    n = len(lead)
    if len(shape) != n + 2 or shape[:n] != lead:
        _bad(f"{name}: shape {tuple(shape)}, expected {tuple(lead)} rows of heads and channels")
    hd = shape[n:]
    if heads is not None and hd != heads:
        _bad(f"{name}: {hd[0]} heads of {hd[1]} channels, expected {heads[0]} of {heads[1]}")
    h, c = hd
    if t.is_contiguous():
        return hd, h * c
    st = t.stride()
    if (c > 1 and st[n + 1] != 1) or (h > 1 and st[n] != c):
        _bad(f"{name}: heads and channels must be contiguous (strides {st})")
    rows = shape[n - 1]
    ld = st[n - 1] if rows > 1 else st[0] if n == 2 and shape[0] > 1 else h * c
    if n == 2 and shape[0] > 1 and st[0] != rows * ld:
        _bad(f"{name}: sequences must follow one another (strides {st})")
    return hd, ld


# What _setup found for contiguous inputs of these shapes and types: it goes by
# them alone, and checking a small call again costs as much as launching it.
_plans: dict = {}


def _setup(q, k, v, log_decay, scale, seq_start, device, step=False):
    """Checks the inputs; returns (dims, leading shape, v's heads, LinattnIn)."""
    starts, S = None, 0
    if seq_start is not None:
        S = seq_start.numel() - 1 if isinstance(seq_start, torch.Tensor) else 0
        if S < 1:
            _bad("seq_start: expected an int32 tensor of at least two offsets")
        starts = _dense(seq_start, "seq_start", (S + 1,), device, torch.int32)
    if type(scale) is not float:
        scale = float(scale)
    io = q.dtype
    key = None
    try:
        if (k.get_device() == v.get_device() == log_decay.get_device() == device and k.dtype is io and v.dtype is io
                and log_decay.dtype is torch.float32 and q.is_contiguous() and k.is_contiguous()
                and v.is_contiguous() and log_decay.is_contiguous()):
            key = (q.shape, k.shape, v.shape, log_decay.shape, io, scale, S, step)
    except AttributeError:
        pass  # not a tensor: refused below by name
    plan = _plans.get(key) if key is not None else None
    if plan is None:
        plan = _check_inputs(q, k, v, log_decay, scale, S, device, step)
        if key is not None:
            if len(_plans) >= 256:
                _plans.clear()
            _plans[key] = plan
    dims, lead, hv, ldq, ldk, ldv = plan
    return dims, lead, hv, LinattnIn(q.data_ptr(), k.data_ptr(), v.data_ptr(), ldq, ldk, ldv, log_decay.data_ptr(),
                                     starts, None)


def _check_inputs(q, k, v, log_decay, scale, packed, device, step):
    io = q.dtype
    if io not in _IO:
        _bad(f"q: dtype {io}, expected bfloat16 or float32")
    nd = q.dim()
    if nd != 3 and (nd != 4 or step):
        _bad(f"q: {nd} dimensions")
    if packed and nd != 3:
        _bad("seq_start goes with packed tokens [T, H, d]")
    lead = q.shape[:-2]
    hk, ldq = _rows(q, "q", lead, device, io)
    _, ldk = _rows(k, "k", lead, device, io, hk)
    hv, ldv = _rows(v, "v", lead, device, io)
    T, S = q.shape[0], packed or 1
    if nd == 4:
        S, T = T, T * q.shape[1]
    if T < 1 or hk[0] < 1 or hv[0] < 1:
        _bad("no tokens or no heads")
    _gpu(log_decay, "log_decay", device, torch.float32)
    tokens = log_decay.dim() != 1
    _dense(log_decay, "log_decay", lead + hv[:1] if tokens else hv[:1], device, torch.float32)
    dims = LinattnDims(T, S, hk[0], hv[0], hk[1], hv[1], _IO[io], 1 if tokens else 0, scale)
    return dims, lead, hv, ldq, ldk, ldv


_sizes: dict = {}


def _ws_bytes(dims, grads, wanted) -> int:
    """linattn_workspace_bytes, remembered by the sizes it follows from."""
    key = (dims.T, dims.S, dims.Hk, dims.Hv, dims.dk, dims.dv, dims.io, dims.decay_tokens, wanted)
    n = _sizes.get(key)
    if n is None:
        n = linattn_workspace_bytes(dims, grads)
        if len(_sizes) >= 256:
            _sizes.clear()
        _sizes[key] = n
    return n


def linattn_workspace_bytes(dims: LinattnDims, grads: LinattnGrads | None = None) -> int:
    """Workspace of linattn_forward, or of linattn_grad for the outputs set in grads."""
    n = ctypes.c_size_t(0)
    _check(lib.ssm_linattn_workspace_bytes(ctypes.byref(dims), None if grads is None else ctypes.byref(grads),
                                           ctypes.byref(n)), "ssm_linattn_workspace_bytes")
    return n.value


def _workspace(ws, nbytes: int, device):
    if ws is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None
    _gpu(ws, "workspace", device, torch.uint8)
    if not ws.is_contiguous() or ws.numel() < nbytes:
        raise SsmError(2, f"workspace: {nbytes} contiguous bytes needed")
    return ws


def _ws_args(w):
    return (None, 0) if w is None else (w.data_ptr(), w.numel())


def linattn_forward(q, k, v, log_decay, seq_start=None, h0=None, scale=1.0, want_state=False, y=None, hT=None,
                    ws=None, stream=None):
    """Runs ssm_linattn_forward; returns (y, hT), hT None unless want_state or
    given.  y has v's shape; hT may be h0.  With seq_start, rows of y outside
    the sequences are not written."""
    device = _gpu(q, "q")
    if stream is not None or device != _current_device():
        with _on(device, stream):
            return linattn_forward(q, k, v, log_decay, seq_start, h0, scale, want_state, y, hT, ws)
    dims, lead, hv, ins = _setup(q, k, v, log_decay, scale, seq_start, device)
    states = (dims.S, dims.Hv, dims.dk, dims.dv)
    ins.h0 = _dense(h0, "h0", states, device, torch.float32)
    if y is None:
        y = torch.empty_like(v) if v.is_contiguous() else torch.empty(v.shape, dtype=v.dtype, device=v.device)
        ldy = hv[0] * hv[1]
    else:
        _, ldy = _rows(y, "y", lead, device, q.dtype, hv)
    if hT is None and want_state:
        hT = torch.empty(states, dtype=torch.float32, device=q.device)
    end = _dense(hT, "hT", states, device, torch.float32)
    w, n = _ws_args(_workspace(ws, _ws_bytes(dims, None, None), device))
    _check(lib.ssm_linattn_forward(ctypes.byref(dims), ctypes.byref(ins), y.data_ptr(), ldy, end, w, n,
                                   _raw_stream(device)), "ssm_linattn_forward")
    return y, hT


def linattn_grad(q, k, v, log_decay, dy, seq_start=None, h0=None, dhT=None, scale=1.0, want=None, grads=None, ws=None,
                 stream=None) -> dict:
    """Runs ssm_linattn_grad; returns the gradient dict.  want: names among
    GRADS (default: all, dh0 only with an h0).  grads: output tensors by
    name (then they alone are computed)."""
    device = _gpu(q, "q")
    if stream is not None or device != _current_device():
        with _on(device, stream):
            return linattn_grad(q, k, v, log_decay, dy, seq_start, h0, dhT, scale, want, grads, ws)
    dims, lead, hv, ins = _setup(q, k, v, log_decay, scale, seq_start, device)
    states = (dims.S, dims.Hv, dims.dk, dims.dv)
    ins.h0 = _dense(h0, "h0", states, device, torch.float32)
    end = _dense(dhT, "dhT", states, device, torch.float32)
    _, lddy = _rows(dy, "dy", lead, device, q.dtype, hv)
    like = {"dq": (q.shape, q.dtype), "dk": (k.shape, q.dtype), "dv": (v.shape, q.dtype),
            "dlog_decay": (log_decay.shape, torch.float32), "dh0": (states, torch.float32)}
    names = grads if grads is not None else want if want is not None else GRADS if h0 is not None else GRADS[:4]
    for name in names:
        if name not in like:
            _bad(f"gradient {name!r} is none of {GRADS}")
    if grads is None:
        grads = {name: torch.empty(like[name][0], dtype=like[name][1], device=q.device) for name in names}
    g = LinattnGrads(*(_dense(grads.get(name), name, like[name][0], device, like[name][1]) for name in GRADS))
    w, n = _ws_args(_workspace(ws, _ws_bytes(dims, g, tuple(name for name in GRADS if grads.get(name) is not None)), device))
    _check(lib.ssm_linattn_grad(ctypes.byref(dims), ctypes.byref(ins), dy.data_ptr(), lddy, end, ctypes.byref(g), w, n,
                                _raw_stream(device)), "ssm_linattn_grad")
    return grads


def linattn_step(q, k, v, log_decay, state, scale=1.0, y=None, stream=None):
    """Runs ssm_linattn_step: row t of q, k [B, Hk, dk] and v [B, Hv, dv] is
    the next token of the sequence with state[t] ([B, Hv, dk, dv], updated in
    place).  Returns y [B, Hv, dv]."""
    device = _gpu(q, "q")
    if stream is not None or device != _current_device():
        with _on(device, stream):
            return linattn_step(q, k, v, log_decay, state, scale, y)
    dims, lead, hv, ins = _setup(q, k, v, log_decay, scale, None, device, step=True)
    if state is None:
        _bad("state is required")
    st = _dense(state, "state", (dims.T, dims.Hv, dims.dk, dims.dv), device, torch.float32)
    if y is None:
        y = torch.empty_like(v) if v.is_contiguous() else torch.empty(v.shape, dtype=v.dtype, device=v.device)
        ldy = hv[0] * hv[1]
    else:
        _, ldy = _rows(y, "y", lead, device, q.dtype, hv)
    _check(lib.ssm_linattn_step(ctypes.byref(dims), ctypes.byref(ins), st, y.data_ptr(), ldy, _raw_stream(device)),
           "ssm_linattn_step")
    return y
