"""Cases of the decayed linear attention, the normalised residual update and
the gradient clipping: their inputs, their plain forms and their definitions.

`run` computes one pass: in plain torch operations where `own` is false,
through adjoint_gradients_amd where it is true.  `exact` computes the same
outputs from the operator's definition in 64 bits.

Operators (op of a case):
  forward    y_t = scale q_t h_t with h_t = e^{g_t} h_{t-1} + k_t v_t^T, per head
  grad       the gradient of L = sum_t <dy_t, y_t> + <dhT, h_T>
  step       one token for each of T sequences, the states updated in place
  norm       r' = r + y, x = io(gamma r' / rms(r'))
  norm_grad  its gradient
  clip       the global norm of many tensors, and the tensors scaled to it
"""
import math
import random

import torch

own = False

_IO = {"f32": torch.float32, "bf16": torch.bfloat16}
_CHUNK = 64  # tokens a chunk of the plain form
_EPS = 1e-5


# ------------------------------------------------------------------ cases

def _attn(name, op, io, T, S, Hk, Hv, dk, dv, decay="token", states=False):
    return {"name": name, "op": op, "io": io, "T": T, "S": S, "Hk": Hk, "Hv": Hv, "dk": dk, "dv": dv,
            "decay": decay, "states": states}


def listed():
    return [
        # one short prompt, fp32: latency, odd length, heads narrower than a tile
        _attn("forward_short", "forward", "f32", 37, 1, 4, 4, 40, 64, states=True),
        # a ragged batch of prompts on 2048 channels (16 heads of 128), states kept for decoding
        _attn("forward_ragged", "forward", "bf16", 16411, 24, 16, 16, 128, 128, states=True),
        # one long document on 1536 channels (24 heads of 64), q and k shared by all heads,
        # a fixed decay for each head
        _attn("forward_long", "forward", "bf16", 131072, 1, 1, 24, 64, 64, decay="head"),
        # gradient in fp32 over a few short sequences, with a state coming in and one going out
        _attn("grad_short", "grad", "f32", 517, 3, 2, 4, 64, 32, states=True),
        # the gradient of one long sequence on 2048 channels
        _attn("grad_long", "grad", "bf16", 65536, 1, 16, 16, 128, 128),
        # decoding for one user
        _attn("step_one", "step", "bf16", 1, 1, 16, 16, 128, 128),
        # decoding for a batch: the states are the traffic
        _attn("step_batch", "step", "bf16", 192, 1, 8, 16, 128, 128),
        # residual update and norm of a decoding batch: latency
        {"name": "norm_rows", "op": "norm", "io": "bf16", "T": 5, "P": 2048},
        # the same over a training batch
        {"name": "norm_train", "op": "norm", "io": "bf16", "T": 65536, "P": 2048},
        # gradient of the norm on 1536 channels
        {"name": "norm_grad_train", "op": "norm_grad", "io": "bf16", "T": 65536, "P": 1536},
        # clipping the gradients of one small layer, and of 12 layers of 2048 channels
        {"name": "clip_layer", "op": "clip", "io": "f32", "layers": 1, "P": 97, "N": 16},
        {"name": "clip_stack", "op": "clip", "io": "f32", "layers": 12, "P": 2048, "N": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("forward", "forward", "grad", "grad", "step", "norm", "norm_grad", "clip"))
    io = rng.choice(("f32", "bf16", "bf16"))
    if op in ("forward", "grad", "step"):
        group = rng.choice((1, 1, 2, 4, 24))
        Hk = 1 if group == 24 else rng.choice((1, 2, 5, 8, 16))
        Hv = Hk * group
        dk, dv = 8 * rng.randint(1, 16), 8 * rng.randint(1, 16)
        if rng.random() < 0.5:
            dk = dv = rng.choice((64, 128))
        # never more work than the long gradient or the batched step
        cap = {"forward": 65536 * 16 * 128 * 128, "grad": 32768 * 16 * 128 * 128, "step": 192 * 16 * 128 * 128}[op]
        T = _log_int(rng, 1, max(1, min({"forward": 131072, "grad": 65536, "step": 256}[op], cap // (Hv * dk * dv))))
        S = 1 if op == "step" else min(T, rng.choice((1, 1, 2, 5, 19, 64)))
        return {"op": op, "io": io, "T": T, "S": S, "Hk": Hk, "Hv": Hv, "dk": dk, "dv": dv,
                "decay": rng.choice(("token", "token", "head")), "states": rng.random() < 0.5}
    if op == "clip":
        return {"op": "clip", "io": rng.choice(("f32", "f32", "bf16")), "layers": rng.randint(1, 12),
                "P": _log_int(rng, 16, 2048), "N": rng.choice((4, 16, 64))}
    P = _log_int(rng, 17, 8192)
    return {"op": op, "io": io, "T": _log_int(rng, 1, max(1, min(65536, 65536 * 1536 // P))), "P": P}


def _lengths(case):
    """Token counts of the packed sequences: ragged, fixed by the case's sizes."""
    T, S = case["T"], case["S"]
    if S == 1:
        return [T]
    rng = random.Random(T * 1009 + S)
    w = [rng.expovariate(1.0) for _ in range(S)]
    n = [int(T * x / sum(w)) for x in w]
    n[rng.randrange(S)] += T - sum(n)
    return n


def _tensors(case):
    """Shapes of the clipped gradients: each layer's weight, decay and bias gradients."""
    P, N = case["P"], case["N"]
    return [(P, P), (N, P), (N, P), (P, N), (P,)] * case["layers"]


# ------------------------------------------------------------------ inputs

def _randn(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    io = _IO[case["io"]]
    st = {"case": case}
    if case["op"] == "clip":
        # gradients an optimiser would have to clip: the norm is above 1
        st["grads"] = [_randn(gen, *s, scale=0.02, dtype=io) for s in _tensors(case)]
        st["out"] = [torch.empty_like(g) for g in st["grads"]]
        return st
    if case["op"] in ("norm", "norm_grad"):
        T, P = case["T"], case["P"]
        st["norm_scale"] = 1.0 + _randn(gen, P, scale=0.1)
        st["r"] = _randn(gen, T, P, scale=2.0)
        if case["op"] == "norm":
            st["y"] = _randn(gen, T, P, dtype=io)
        else:
            r64 = st["r"].double()
            st["rinv"] = torch.rsqrt((r64 * r64).mean(1) + _EPS).float()
            st["dx"] = _randn(gen, T, P, dtype=io)
            st["dr"] = _randn(gen, T, P)
        return st
    T, Hk, Hv, dk, dv = (case[n] for n in ("T", "Hk", "Hv", "dk", "dv"))
    st["q"] = _randn(gen, T, Hk, dk, dtype=io)
    st["k"] = _randn(gen, T, Hk, dk, dtype=io)
    st["v"] = _randn(gen, T, Hv, dv, dtype=io)
    st["scale"] = dk ** -0.5
    if case["decay"] == "token":
        # -alpha_h softplus(z + bias_h), softplus(bias_h) in 1e-3 .. 1e-1, alpha_h in 1 .. 16
        u = torch.rand(Hv, generator=gen, device="cuda") * 0.099 + 0.001
        bias = torch.log(torch.expm1(u))
        alpha = 1.0 + torch.arange(Hv, device="cuda", dtype=torch.float32) % 16
        z = _randn(gen, T, Hv, scale=0.5)
        st["log_decay"] = -alpha * torch.nn.functional.softplus(z + bias)
    else:
        # decays of 1 - 2^-1 .. 1 - 2^-9 over the heads
        e = 1.0 + 8.0 * torch.rand(Hv, generator=gen, device="cuda")
        st["log_decay"] = torch.log1p(-torch.exp2(-e))
    if case["op"] == "step":
        st["state"] = _randn(gen, T, Hv, dk, dv)
        return st
    n = _lengths(case)
    st["lengths"] = n
    st["seq_start"] = None
    if case["S"] > 1:
        edges = [0]
        for c in n:
            edges.append(edges[-1] + c)
        st["seq_start"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
    st["h0"] = _randn(gen, case["S"], Hv, dk, dv) if case["states"] else None
    if case["op"] == "grad":
        st["dy"] = _randn(gen, T, Hv, dv, dtype=io)
        st["dhT"] = _randn(gen, case["S"], Hv, dk, dv) if case["states"] else None
    return st


# ------------------------------------------------------------------ the framework's calls

def _run_own(st):
    import adjoint_gradients_amd as agm

    case = st["case"]
    op = case["op"]
    if op == "forward":
        y, hT = agm.linattn_forward(st["q"], st["k"], st["v"], st["log_decay"], seq_start=st["seq_start"],
                                    h0=st["h0"], scale=st["scale"], want_state=case["states"])
        return (y, hT) if case["states"] else (y,)
    if op == "grad":
        g = agm.linattn_grad(st["q"], st["k"], st["v"], st["log_decay"], st["dy"], seq_start=st["seq_start"],
                             h0=st["h0"], dhT=st["dhT"], scale=st["scale"])
        out = (g["dq"], g["dk"], g["dv"], g["dlog_decay"])
        return out + (g["dh0"],) if case["states"] else out
    if op == "step":
        y = agm.linattn_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], scale=st["scale"])
        return y, st["state"]
    if op == "norm":
        x, r, rinv = agm.add_norm(st["r"], st["y"], st["norm_scale"], eps=_EPS)
        return x, r, rinv
    if op == "norm_grad":
        dr, dscale = agm.add_norm_grad(st["r"], st["rinv"], st["norm_scale"], st["dx"], st["dr"])
        return dr, dscale
    norm = agm.clip_grads(st["grads"], 1.0, out=st["out"])
    return tuple(st["out"]) + (norm,)


# ------------------------------------------------------------------ plain forms

def _heads(t, Hv):
    """[T, Hk, d] as float32 [T, Hv, d]: every value head's own copy."""
    t = t.float()
    return t if t.shape[1] == Hv else t.repeat_interleave(Hv // t.shape[1], dim=1)


def _chunks(t, pos, nc):
    """Packed tokens [T, H, ...] into zero-padded chunks [nc, H, C, ...]."""
    out = t.new_zeros((nc * _CHUNK,) + tuple(t.shape[1:]))
    out[pos] = t
    out = out.view((nc, _CHUNK) + tuple(t.shape[1:]))
    return out.transpose(1, 2).contiguous()


def _tokens(t, pos):
    """The reverse of _chunks."""
    t = t.transpose(1, 2).contiguous()
    return t.view((-1,) + tuple(t.shape[2:]))[pos]


def _layout(st):
    """Padded position of each token, chunk count, first chunk and chunk count of each sequence."""
    pos, spans, c0 = [], [], 0
    for n in st["lengths"]:
        pos.append(torch.arange(n, device="cuda") + c0 * _CHUNK)
        nc = (n + _CHUNK - 1) // _CHUNK
        spans.append((c0, nc))
        c0 += nc
    return torch.cat(pos), c0, spans


def _plain_chunks(st):
    """What the plain forward pass and gradient share: chunks, decays, entering states."""
    case = st["case"]
    T, Hv = case["T"], case["Hv"]
    pos, nc, spans = _layout(st)
    g = st["log_decay"].double()
    g = g if case["decay"] == "token" else g.expand(T, Hv)
    G = _chunks(g, pos, nc).cumsum(-1)  # [nc, H, C]; padding decays by 1
    causal = torch.ones(_CHUNK, _CHUNK, dtype=torch.bool, device="cuda").tril()
    D = torch.where(causal, (G.unsqueeze(-1) - G.unsqueeze(-2)), -math.inf).exp().float()
    wq = G.exp().float().unsqueeze(-1)
    wk = (G[..., -1:] - G).exp().float().unsqueeze(-1)
    wc = G[..., -1].exp().float()[..., None, None]
    q, k, v = (_chunks(_heads(st[n], Hv), pos, nc) for n in ("q", "k", "v"))
    U = (k * wk).transpose(-1, -2).contiguous() @ v
    S_in = torch.empty_like(U)
    last = []
    for s, (c0, n) in enumerate(spans):
        h = st["h0"][s].clone() if st["h0"] is not None else torch.zeros_like(U[0]) if nc else None
        for c in range(c0, c0 + n):
            S_in[c] = h
            h = h * wc[c] + U[c]
        last.append(h)
    return pos, nc, spans, q, k, v, G, D, wq, wk, wc, S_in, last


def _plain_forward(st):
    case = st["case"]
    pos, nc, spans, q, k, v, G, D, wq, wk, wc, S_in, last = _plain_chunks(st)
    scores = (q @ k.transpose(-1, -2).contiguous()) * D
    y = (scores @ v + (q * wq) @ S_in) * st["scale"]
    y = _tokens(y, pos).to(_IO[case["io"]])
    return (y, torch.stack(last)) if case["states"] else (y,)


def _group_sum(t, Hk):
    T, Hv, d = t.shape
    return t if Hv == Hk else t.view(T, Hk, Hv // Hk, d).sum(2)


def _plain_grad(st):
    case = st["case"]
    io, Hk, sc = _IO[case["io"]], case["Hk"], st["scale"]
    pos, nc, spans, q, k, v, G, D, wq, wk, wc, S_in, last = _plain_chunks(st)
    dy = _chunks(st["dy"].float(), pos, nc) * sc
    V = (q * wq).transpose(-1, -2).contiguous() @ dy
    D_out = torch.empty_like(V)
    first = []
    for s, (c0, n) in enumerate(spans):
        d = st["dhT"][s].clone() if st["dhT"] is not None else torch.zeros_like(V[0])
        for c in range(c0 + n - 1, c0 - 1, -1):
            D_out[c] = d
            d = d * wc[c] + V[c]
        first.append(d)
    P = (q @ k.transpose(-1, -2).contiguous()) * D
    dP = (dy @ v.transpose(-1, -2).contiguous()) * D
    dq_in = wq * (dy @ S_in.transpose(-1, -2).contiguous())
    dk_out = wk * (v @ D_out.transpose(-1, -2).contiguous())
    dq = dP @ k + dq_in
    dk = dP.transpose(-1, -2).contiguous() @ q + dk_out
    dv = P.transpose(-1, -2).contiguous() @ dy + wk * (k @ D_out)
    # d log_decay of token t: what passes from a token j < t to a token i >= t, for i and j inside
    # or outside t's chunk; sums in 64 bits
    M = (dP * (q @ k.transpose(-1, -2).contiguous())).tril(-1).double()
    R, Cc = (q.double() * dq_in.double()).sum(-1), (k.double() * dk_out.double()).sum(-1)
    x = (R + M.sum(-1) - M.sum(-2)).flip(-1).cumsum(-1).flip(-1) + Cc.cumsum(-1) - Cc
    x = x + (S_in.double() * D_out.double()).sum((-1, -2)).unsqueeze(-1) * G[..., -1:].exp()
    dg = _tokens(x.unsqueeze(-1), pos).squeeze(-1)
    if case["decay"] == "head":
        dg = dg.sum(0)
    out = (_group_sum(_tokens(dq, pos), Hk).to(io), _group_sum(_tokens(dk, pos), Hk).to(io),
           _tokens(dv, pos).to(io), dg.float())
    return out + (torch.stack(first),) if case["states"] else out


def _plain_step(st):
    Hv = st["case"]["Hv"]
    q, k, v = _heads(st["q"], Hv), _heads(st["k"], Hv), st["v"].float()
    a = st["log_decay"].exp()
    a = a if a.dim() == 2 else a.unsqueeze(0)
    h = st["state"]
    h.mul_(a[..., None, None])
    h.add_(k.unsqueeze(-1) * v.unsqueeze(-2))
    y = (q.unsqueeze(-1) * h).sum(-2) * st["scale"]
    return y.to(st["q"].dtype), h


def _plain_norm(st):
    r = st["r"] + st["y"].float()
    rinv = torch.rsqrt((r * r).mean(1) + _EPS)
    return (st["norm_scale"] * (r * rinv[:, None])).to(st["y"].dtype), r, rinv


def _plain_norm_grad(st):
    xh = st["r"] * st["rinv"][:, None]
    dx = st["dx"].float()
    u = st["norm_scale"] * dx
    m = (u * xh).mean(1, keepdim=True)
    return st["dr"] + st["rinv"][:, None] * (u - xh * m), (dx * xh).sum(0, dtype=torch.float64).float()


def _plain_clip(st):
    total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt()
    coef = torch.where(total > 1.0, 1.0 / total, torch.ones_like(total)).float()
    for g, o in zip(st["grads"], st["out"]):
        o.copy_(g.float() * coef)
    return tuple(st["out"]) + (total.float().view(1),)


_PLAIN = {"forward": _plain_forward, "grad": _plain_grad, "step": _plain_step, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad, "clip": _plain_clip}


def run(state):
    return _run_own(state) if own else _PLAIN[state["case"]["op"]](state)


# ------------------------------------------------------------------ work

def work(case):
    es = 2 if case["io"] == "bf16" else 4
    op = case["op"]
    if op == "clip":
        n = sum(math.prod(s) for s in _tensors(case))
        return {"bytes": 2 * es * n + 4, "flops": 3 * n}
    T = case["T"]
    if op in ("norm", "norm_grad"):
        n = T * case["P"]
        if op == "norm":
            return {"bytes": n * (4 + es + 4 + es) + 4 * T + 4 * case["P"], "flops": 5 * n}
        return {"bytes": n * (4 + es + 4 + 4) + 4 * T + 8 * case["P"], "flops": 10 * n}
    Hk, Hv, dk, dv = (case[n] for n in ("Hk", "Hv", "dk", "dv"))
    qk, vy = T * Hk * dk * es, T * Hv * dv * es
    gd = 4 * (T * Hv if case["decay"] == "token" else Hv)
    mat = Hv * dk * dv
    if op == "step":
        return {"bytes": 2 * qk + 2 * vy + gd + 8 * T * mat, "flops": 5 * T * mat}
    states = 4 * case["S"] * mat if case["states"] else 0
    if op == "forward":
        return {"bytes": 2 * qk + 2 * vy + gd + 2 * states, "flops": 4 * T * mat}
    return {"bytes": 4 * qk + 3 * vy + 2 * gd + 3 * states, "flops": 10 * T * mat}


# ------------------------------------------------------------------ definitions in 64 bits

def _rows(t, lengths, Hv=None):
    """Packed [T, H, ...] -> [Lmax, S, Hv, ...] in 64 bits, zeros behind each sequence."""
    t = t.double()
    if Hv is not None and t.shape[1] != Hv:
        t = t.repeat_interleave(Hv // t.shape[1], dim=1)
    out = t.new_zeros((max(lengths), len(lengths)) + tuple(t.shape[1:]))
    t0 = 0
    for s, n in enumerate(lengths):
        out[:n, s] = t[t0:t0 + n]
        t0 += n
    return out


def _packed(t, lengths):
    return torch.cat([t[:n, s] for s, n in enumerate(lengths)])


def _exact_attn(st):
    """The recurrence, one token at a time; sequences that have ended stand still."""
    case, n = st["case"], st["lengths"]
    T, S, Hk, Hv, dk, dv = (case[x] for x in ("T", "S", "Hk", "Hv", "dk", "dv"))
    sc = st["scale"]
    q, k, v = _rows(st["q"], n, Hv) * sc, _rows(st["k"], n, Hv), _rows(st["v"], n)
    g = st["log_decay"]
    # beyond a sequence's end: log decay 0 and k = 0, so the state stays
    a = _rows(g if case["decay"] == "token" else g.expand(T, Hv), n).exp()[..., None, None]
    L = max(n)
    h = st["h0"].double() if st["h0"] is not None else torch.zeros(S, Hv, dk, dv, dtype=torch.float64, device="cuda")
    grad = case["op"] == "grad"
    src = _rows(st["dy"], n) if grad else None
    res = torch.empty(L, S, Hv, dk if grad else dv, dtype=torch.float64, device="cuda")
    for t in range(L):
        h = a[t] * h + k[t].unsqueeze(-1) * v[t].unsqueeze(-2)
        if grad:
            res[t] = (h * src[t].unsqueeze(-2)).sum(-1) * sc
        else:
            res[t] = (h * q[t].unsqueeze(-1)).sum(-2)
    if not grad:
        y = _packed(res, n)
        return (y, h) if case["states"] else (y,)
    dq = res
    m = st["dhT"].double() if st["dhT"] is not None else torch.zeros_like(h)
    tail = (h * m).sum((-1, -2))
    dkk = torch.empty_like(dq)
    dvv = torch.empty(L, S, Hv, dv, dtype=torch.float64, device="cuda")
    for t in range(L - 1, -1, -1):
        m = m + q[t].unsqueeze(-1) * src[t].unsqueeze(-2)
        dkk[t] = (m * v[t].unsqueeze(-2)).sum(-1)
        dvv[t] = (m * k[t].unsqueeze(-1)).sum(-2)
        m = a[t] * m
    x = ((q / sc) * dq).sum(-1) - (k * dkk).sum(-1)
    dg = _packed(tail + x.flip(0).cumsum(0).flip(0), n)
    if case["decay"] == "head":
        dg = dg.sum(0)
    out = (_group_sum(_packed(dq, n), Hk), _group_sum(_packed(dkk, n), Hk), _packed(dvv, n), dg)
    return out + (m,) if case["states"] else out


def exact(case, seed):
    op = case["op"]
    if op in ("forward", "grad"):
        # one launch after the other for each token of the longest sequence
        if max(_lengths(case)) > 140000:
            return None
        return _exact_attn(prepare(case, seed))
    st = prepare(case, seed)
    if op == "step":
        Hv = case["Hv"]
        q, k, v = (st[x].double() for x in ("q", "k", "v"))
        if case["Hk"] != Hv:
            q, k = (x.repeat_interleave(Hv // case["Hk"], dim=1) for x in (q, k))
        a = st["log_decay"].double().exp().expand(case["T"], Hv)
        h = a[..., None, None] * st["state"].double() + k.unsqueeze(-1) * v.unsqueeze(-2)
        return (h * q.unsqueeze(-1)).sum(-2) * st["scale"], h
    if op == "norm":
        r = st["r"].double() + st["y"].double()
        rinv = (r.square().sum(1) / case["P"] + _EPS) ** -0.5
        return r * rinv[:, None] * st["norm_scale"].double(), r, rinv
    if op == "norm_grad":
        ri = st["rinv"].double()[:, None]
        xh, dx, gm = st["r"].double() * ri, st["dx"].double(), st["norm_scale"].double()
        m = (gm * dx * xh).sum(1, keepdim=True) / case["P"]
        return st["dr"].double() + ri * (gm * dx - xh * m), (dx * xh).sum(0)
    total = math.fsum(float(g.double().square().sum()) for g in st["grads"]) ** 0.5
    coef = 1.0 / total if total > 1.0 else 1.0
    return tuple(g.double() * coef for g in st["grads"]) + (torch.tensor([total], dtype=torch.float64, device="cuda"),)
