"""64-bit reference of the decayed linear attention, one token at a time, and
the tolerances of the GPU tests.

Tolerances count roundings.  A value rounded to bf16 is off by at most half a
step, 2^-8 of itself.  A bf16 output has that one rounding, whose mean square
is at most 2^-8; its operands that are not bf16 (decayed scores, state,
weighted v) keep two bf16 parts, 2^-17 of them, and two such operands meet at
most.  What is fp32 but made from bf16 inputs keeps three parts of each; its
bound, 2^-16 in the mean square, would hold with two.  In fp32 a result of n
sums is off by about sqrt(n) 2^-24, n a few thousand here: 2^-18."""
import numpy as np
import torch

RMS = {("bf16", torch.bfloat16): 2.0 ** -8, ("bf16", torch.float32): 2.0 ** -16,
       ("f32", torch.float32): 2.0 ** -18}


def rms_err(got, ref):
    d = float((got.double().cpu() - ref).square().mean().sqrt()) if ref.numel() else 0.0
    n = float(ref.square().mean().sqrt()) if ref.numel() else 0.0
    return d / n if n else d


def forward(q, k, v, g, spans, scale, h0=None):
    """y [T, Hv, dv] (zeros outside the spans) and the final states, in float64."""
    T, Hv, dv = v.shape
    G = Hv // q.shape[1]
    q, k = (x.repeat_interleave(G, dim=1) for x in (q, k))
    g = g if g.dim() == 2 else g.expand(T, Hv)
    ys, ends = [None] * T, []
    for s, (a, b) in enumerate(spans):
        h = h0[s] if h0 is not None else torch.zeros(Hv, q.shape[2], dv, dtype=torch.float64)
        for t in range(a, b):
            h = torch.exp(g[t])[:, None, None] * h + k[t][:, :, None] * v[t][:, None, :]
            ys[t] = scale * (q[t][:, :, None] * h).sum(1)
        ends.append(h)
    z = torch.zeros(Hv, dv, dtype=torch.float64)
    return torch.stack([z if y is None else y for y in ys]), torch.stack(ends)


def gradient(q, k, v, g, dy, spans, scale, h0=None, dhT=None):
    """The gradients of L by reverse mode through `forward`, and L."""
    xs = {"dq": q, "dk": k, "dv": v, "dlog_decay": g}
    if h0 is not None:
        xs["dh0"] = h0
    xs = {n: x.clone().requires_grad_(True) for n, x in xs.items()}
    y, hT = forward(xs["dq"], xs["dk"], xs["dv"], xs["dlog_decay"], spans, scale, xs.get("dh0"))
    mask = torch.zeros(v.shape[0], dtype=torch.bool)
    for a, b in spans:
        mask[a:b] = True
    L = (dy[mask] * y[mask]).sum()
    if dhT is not None:
        L = L + (dhT * hT).sum()
    grads = torch.autograd.grad(L, list(xs.values()), allow_unused=True)
    return {n: torch.zeros_like(x) if d is None else d for (n, x), d in zip(xs.items(), grads)}, L.detach()


def inputs(seed, T, Hk, Hv, dk, dv, io, decay="token", S=1, states=False):
    """Float64 CPU inputs that the io dtype holds exactly; log decays of -1e-3 .. -2 over the heads."""
    rng = np.random.default_rng(seed)

    def r(*shape):
        x = torch.from_numpy(rng.standard_normal(shape).astype(np.float32))
        return (x.to(torch.bfloat16) if io == "bf16" else x).double()

    f32 = lambda *shape: torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).double()
    alpha = np.exp(np.linspace(np.log(1e-3), np.log(2.0), Hv))
    u = rng.random((T, Hv) if decay == "token" else (Hv,))
    d = {"q": r(T, Hk, dk), "k": r(T, Hk, dk), "v": r(T, Hv, dv), "dy": r(T, Hv, dv),
         "g": torch.from_numpy((-alpha * (0.5 + u)).astype(np.float32)).double()}
    d["h0"] = f32(S, Hv, dk, dv) if states else None
    d["dhT"] = f32(S, Hv, dk, dv) if states else None
    return d
