"""The operators' C entries and bindings without a GPU: sizes, and refusals
before anything is launched (fake device addresses are never dereferenced)."""
import ctypes
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, ARG, WS, UNSUPPORTED = 0, 1, 2, 4


@pytest.fixture(scope="module")
def agm():
    if not os.path.exists(os.path.join(ROOT, "adjoint_gradients_amd", "libssm_adjoint.so")):
        pytest.fail("libssm_adjoint.so not built (run __graft_entry__.build())")
    import adjoint_gradients_amd as agm

    return agm


A = [0x100000 * (i + 1) for i in range(16)]  # aligned, never dereferenced


def dims(agm, T=100, S=1, Hk=2, Hv=4, dk=64, dv=64, io=1, tokens=1, scale=1.0):
    return agm.LinattnDims(T, S, Hk, Hv, dk, dv, io, tokens, scale)


def ins(agm, **kw):
    d = dict(q=A[0], k=A[1], v=A[2], ldq=128, ldk=128, ldv=256, log_decay=A[3], seq_start=None, h0=None)
    d.update(kw)
    return agm.LinattnIn(**d)


def size(agm, d, g=None):
    n = ctypes.c_size_t(7)
    rc = agm.lib.ssm_linattn_workspace_bytes(ctypes.byref(d), None if g is None else ctypes.byref(g), ctypes.byref(n))
    return rc, n.value


def forward(agm, d, i, y=A[4], ldy=256, hT=None, ws=A[5], nbytes=1 << 40):
    return agm.lib.ssm_linattn_forward(ctypes.byref(d), ctypes.byref(i), y, ldy, hT, ws, nbytes, None)


def grad(agm, d, i, g, dy=A[4], lddy=256, dhT=None, ws=A[5], nbytes=1 << 40):
    return agm.lib.ssm_linattn_grad(ctypes.byref(d), ctypes.byref(i), dy, lddy, dhT, ctypes.byref(g), ws, nbytes, None)


def step(agm, d, i, state=A[6], y=A[4], ldy=256):
    return agm.lib.ssm_linattn_step(ctypes.byref(d), ctypes.byref(i), state, y, ldy, None)


BAD_DIMS = [(dict(T=0), ARG), (dict(Hk=0), ARG), (dict(Hv=0), ARG), (dict(dk=0), ARG), (dict(dv=-8), ARG),
            (dict(Hk=3), ARG), (dict(scale=float("nan")), ARG), (dict(scale=float("inf")), ARG), (dict(tokens=2), ARG),
            (dict(io=2), UNSUPPORTED), (dict(dk=12), UNSUPPORTED), (dict(dv=136), UNSUPPORTED),
            (dict(Hk=8192, Hv=8192), UNSUPPORTED), (dict(T=1 << 31), UNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_DIMS, ids=[str(b[0]) for b in BAD_DIMS])
def test_linattn_refuses_dims(agm, kw, code):
    d = dims(agm, **kw)
    assert size(agm, d) == (code, 0)
    assert forward(agm, d, ins(agm, ldq=1 << 22, ldk=1 << 22, ldv=1 << 22), ldy=1 << 22) == code
    assert grad(agm, d, ins(agm), agm.LinattnGrads(dq=A[7])) == code
    assert step(agm, d, ins(agm)) == code


@pytest.mark.parametrize("kw,code", [(dict(S=0), ARG), (dict(S=70000, T=70000), UNSUPPORTED),
                                     (dict(S=60000, T=60000, Hk=100, Hv=100), UNSUPPORTED)])
def test_linattn_refuses_sequence_counts(agm, kw, code):
    d = dims(agm, **kw)
    assert size(agm, d) == (code, 0)
    assert forward(agm, d, ins(agm)) == code


BAD_INS = [dict(q=None), dict(k=None), dict(v=None), dict(log_decay=None), dict(q=A[0] + 8), dict(v=A[2] + 4),
           dict(log_decay=A[3] + 4), dict(h0=A[8] + 8), dict(seq_start=A[9] + 4), dict(ldq=120), dict(ldk=129),
           dict(ldv=255), dict(ldv=(1 << 22) + 8)]


@pytest.mark.parametrize("kw", BAD_INS, ids=str)
def test_linattn_refuses_inputs(agm, kw):
    d, i = dims(agm), ins(agm, **kw)
    assert forward(agm, d, i) == ARG
    assert grad(agm, d, i, agm.LinattnGrads(dq=A[7])) == ARG
    assert step(agm, d, i) == ARG


def test_linattn_refuses_the_rest(agm):
    d, i = dims(agm), ins(agm)
    assert forward(agm, d, i, y=None) == ARG and forward(agm, d, i, y=A[4] + 2) == ARG
    assert forward(agm, d, i, ldy=248) == ARG and forward(agm, d, i, hT=A[6] + 8) == ARG
    assert forward(agm, dims(agm, S=3), i) == ARG  # 100 tokens are no three equal sequences
    g = agm.LinattnGrads
    assert grad(agm, d, i, g()) == ARG and size(agm, d, g()) == (ARG, 0)
    assert grad(agm, d, i, g(dk=A[7] + 2)) == ARG and grad(agm, d, i, g(dh0=A[7] + 4)) == ARG
    assert grad(agm, d, i, g(dq=A[7]), dy=None) == ARG and grad(agm, d, i, g(dq=A[7]), lddy=8) == ARG
    assert grad(agm, d, i, g(dq=A[7]), dhT=A[8] + 4) == ARG
    assert step(agm, d, i, state=None) == ARG and step(agm, d, i, y=None) == ARG
    assert step(agm, d, ins(agm, h0=A[8])) == ARG and step(agm, d, ins(agm, seq_start=A[8])) == ARG
    assert step(agm, dims(agm, T=(1 << 22) + 1), i) == UNSUPPORTED


def test_linattn_workspace(agm):
    # few tokens for one sequence: nothing to split, nothing needed
    assert size(agm, dims(agm, T=128)) == (OK, 0)
    rc, n = size(agm, dims(agm, T=65536))
    assert rc == OK and n > 0
    # a long sequence needs its segments' states, however few heads; refused when short or unaligned
    d, i = dims(agm, T=65536), ins(agm)
    assert forward(agm, d, i, nbytes=n - 1) == WS and forward(agm, d, i, ws=None) == WS
    assert forward(agm, d, i, ws=A[5] + 16) == WS
    g = agm.LinattnGrads(dq=A[7], dk=A[8], dv=A[9], dlog_decay=A[10])
    rc, full = size(agm, d, g)
    assert rc == OK and full > n
    assert grad(agm, d, i, g, nbytes=full - 1) == WS
    # without the decay's gradient, and without the sums over shared heads
    rc, less = size(agm, d, agm.LinattnGrads(dq=A[7], dk=A[8], dv=A[9]))
    rc, least = size(agm, d, agm.LinattnGrads(dv=A[9]))
    assert full > less > least > 0
    # the buffers do not grow with the square of anything: 16 times the tokens, at most 16 times the bytes
    rc, big = size(agm, dims(agm, T=1 << 20), g)
    assert big <= 17 * full


def norm_call(agm, T=4, P=64, io=1, r=A[0], y=A[1], scale=A[2], eps=1e-5, r_out=A[3], x=A[4], rinv=A[5]):
    return agm.lib.ssm_add_norm(T, P, io, r, y, scale, eps, r_out, x, rinv, None)


def norm_grad(agm, T=4, P=64, io=1, r=A[0], rinv=A[1], scale=A[2], dx=A[3], dro=A[4], dr=A[5], ds=A[6], ws=A[7],
              nbytes=1 << 30):
    return agm.lib.ssm_add_norm_grad(T, P, io, r, rinv, scale, dx, dro, dr, ds, ws, nbytes, None)


def test_norm_refusals(agm):
    for kw in (dict(T=0), dict(P=0), dict(r=None), dict(scale=None), dict(x=None), dict(r=A[0] + 4), dict(y=A[1] + 2),
               dict(r_out=None), dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(rinv=A[5] + 4)):
        assert norm_call(agm, **kw) == ARG, kw
    for kw in (dict(P=16385), dict(io=2), dict(T=(1 << 31) + 1)):
        assert norm_call(agm, **kw) == UNSUPPORTED, kw
    for kw in (dict(T=0), dict(r=None), dict(rinv=None), dict(scale=None), dict(dx=None), dict(dr=None),
               dict(dro=A[4] + 8), dict(ds=A[6] + 4)):
        assert norm_grad(agm, **kw) == ARG, kw
    assert norm_grad(agm, P=16385) == UNSUPPORTED and norm_grad(agm, io=-1) == UNSUPPORTED
    n = agm.lib.ssm_add_norm_grad_workspace_bytes(4, 64)
    assert n >= 4 * 64 * 4
    assert norm_grad(agm, nbytes=n - 1) == WS and norm_grad(agm, ws=None) == WS and norm_grad(agm, ws=A[7] + 32) == WS
    assert agm.lib.ssm_add_norm_grad_workspace_bytes(0, 64) == 0
    assert agm.lib.ssm_add_norm_grad_workspace_bytes(4, 20000) == 0
    # bounded however many rows
    assert agm.lib.ssm_add_norm_grad_workspace_bytes(1 << 30, 2048) == agm.lib.ssm_add_norm_grad_workspace_bytes(1 << 20, 2048)


def clip(agm, count=2, n=(5, 6), ptrs=(A[0], A[1]), outs=(A[2], A[3]), io=0, max_norm=1.0, norm=A[4], ws=A[5],
         nbytes=1 << 30):
    P, N = (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(n))(*n)
    O = None if outs is None else (ctypes.c_void_p * len(outs))(*outs)
    return agm.lib.ssm_clip_grads(count, P, O, N, io, max_norm, norm, ws, nbytes, None)


def test_clip_refusals(agm):
    for kw in (dict(count=0), dict(count=-1), dict(n=(5, -1)), dict(ptrs=(A[0], None)), dict(ptrs=(A[0] + 8, A[1])),
               dict(outs=(A[2], None)), dict(max_norm=0.0), dict(max_norm=-1.0), dict(max_norm=float("nan")),
               dict(norm=None)):
        assert clip(agm, **kw) == ARG, kw
    assert clip(agm, count=65537, n=(0,) * 65537, ptrs=(None,) * 65537, outs=None) == ARG
    assert clip(agm, io=5) == UNSUPPORTED
    assert clip(agm, ws=None) == WS and clip(agm, nbytes=8) == WS and clip(agm, ws=A[5] + 8) == WS
    one = (ctypes.c_int64 * 1)(3)
    assert agm.lib.ssm_clip_grads_workspace_bytes(1, one) > 0
    assert agm.lib.ssm_clip_grads_workspace_bytes(0, one) == 0 and agm.lib.ssm_clip_grads_workspace_bytes(1, None) == 0


def test_bindings_refuse_host_tensors_and_strangers(agm):
    q = torch.zeros(4, 1, 8)
    for call in (lambda: agm.linattn_forward(q, q, q, torch.zeros(4, 1)),
                 lambda: agm.linattn_grad(q, q, q, torch.zeros(4, 1), q),
                 lambda: agm.linattn_step(q, q, q, torch.zeros(4, 1), torch.zeros(4, 1, 8, 8)),
                 lambda: agm.add_norm(torch.zeros(2, 4), None, torch.ones(4)),
                 lambda: agm.add_norm_grad(torch.zeros(2, 4), torch.ones(2), torch.ones(4), torch.zeros(2, 4)),
                 lambda: agm.clip_grads([torch.zeros(3)], 1.0)):
        with pytest.raises(agm.SsmError, match="GPU tensor"):
            call()
    with pytest.raises(agm.SsmError, match="torch.Tensor"):
        agm.linattn_forward(None, q, q, q)
    with pytest.raises(agm.SsmError, match="no gradients"):
        agm.clip_grads([], 1.0)
