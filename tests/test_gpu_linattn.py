"""The decayed linear attention on the GPU against a 64-bit token-by-token
reference (tests/linattn_ref.py, which derives the tolerances)."""
import pytest
import torch

import linattn_ref as ref
from gpu_util import say

pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def agm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import adjoint_gradients_amd as agm

    return agm


def dev(x, dtype):
    return None if x is None else x.to(dtype).cuda()


def spans_of(lengths, first=0):
    out, t = [], first
    for n in lengths:
        out.append((t, t + n))
        t += n
    return out


def device_inputs(d, io):
    t = {n: dev(d[n], IO[io]) for n in ("q", "k", "v", "dy")}
    t.update({n: dev(d[n], torch.float32) for n in ("g", "h0", "dhT")})
    return t


def starts(spans):
    return torch.tensor([spans[0][0]] + [b for _, b in spans], dtype=torch.int32, device="cuda")


def check(name, got, want, io, what):
    err = ref.rms_err(got, want)
    tol = ref.RMS[io, got.dtype]
    say(f"  {what} {name}: rms error {err:.2e} (<= {tol:.2e})")
    assert err <= tol, (what, name, err)


def covered(spans, T):
    m = torch.zeros(T, dtype=torch.bool)
    for a, b in spans:
        m[a:b] = True
    return m


# lengths, rows before and behind the sequences, heads and widths
CASES = [
    # one token; one chunk less one; whole chunks; one more; several segments
    dict(lens=[1], Hk=1, Hv=1, dk=8, dv=8),
    dict(lens=[63], Hk=2, Hv=2, dk=64, dv=64),
    dict(lens=[64], Hk=1, Hv=2, dk=128, dv=128),
    dict(lens=[65], Hk=1, Hv=1, dk=40, dv=72),
    dict(lens=[700], Hk=1, Hv=2, dk=64, dv=128, states=True),
    dict(lens=[700], Hk=2, Hv=2, dk=128, dv=64, decay="head"),
    # ragged: empty, single and long sequences, rows outside all of them
    dict(lens=[0, 1, 300, 0, 17, 129, 0], Hk=1, Hv=3, dk=16, dv=24, states=True, before=3, behind=5),
    dict(lens=[5, 600, 1], Hk=2, Hv=4, dk=128, dv=128, states=True, decay="head", behind=2),
    dict(lens=[0], Hk=1, Hv=1, dk=64, dv=64, states=True, behind=4),
    # the other padded shapes
    dict(lens=[257, 31], Hk=3, Hv=3, dk=120, dv=56, states=True),
]
IDS = [f"{'+'.join(map(str, c['lens']))}_h{c['Hk']}x{c['Hv']}_d{c['dk']}x{c['dv']}" for c in CASES]


def build(c, io, seed):
    spans = spans_of(c["lens"], c.get("before", 0))
    T = spans[-1][1] + c.get("behind", 0)
    d = ref.inputs(seed, T, c["Hk"], c["Hv"], c["dk"], c["dv"], io, c.get("decay", "token"), len(spans),
                   c.get("states", False))
    return spans, T, d, c["dk"] ** -0.5


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_forward(agm, c, io):
    spans, T, d, scale = build(c, io, 11)
    want, ends = ref.forward(d["q"], d["k"], d["v"], d["g"], spans, scale, d["h0"])
    t = device_inputs(d, io)
    packed = len(spans) > 1 or T != spans[-1][1]
    y = torch.full((T, c["Hv"], c["dv"]), 7.0, dtype=IO[io], device="cuda")
    hT = torch.full_like(dev(ends, torch.float32), float("nan"))
    # rows outside the sequences may hold anything
    out = ~covered(spans, T)
    for n in ("q", "k", "v"):
        t[n][out.cuda()] = float("nan")
    agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=starts(spans) if packed else None, h0=t["h0"],
                        scale=scale, y=y, hT=hT)
    torch.cuda.synchronize()
    y = y.cpu()
    assert bool((y[out] == 7.0).all())
    m = covered(spans, T)
    check("y", y[m], want[m], io, "forward")
    check("hT", hT.cpu(), ends, io, "forward")
    if io == "bf16" and bool(m.any()):
        a, _ = ref.forward(d["q"].abs(), d["k"].abs(), d["v"].abs(), d["g"], spans, scale,
                           None if d["h0"] is None else d["h0"].abs())
        bound = 2.0 ** -8 * (want.abs() + 2 * a) * 1.01
        assert bool(((y.double() - want).abs()[m] <= bound[m] + 1e-30).all())


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("c", CASES, ids=IDS)
def test_gradient(agm, c, io):
    spans, T, d, scale = build(c, io, 12)
    want, _ = ref.gradient(d["q"], d["k"], d["v"], d["g"], d["dy"], spans, scale, d["h0"], d["dhT"])
    t = device_inputs(d, io)
    packed = len(spans) > 1 or T != spans[-1][1]
    out = ~covered(spans, T)
    for n in ("q", "k", "v", "dy"):
        t[n][out.cuda()] = float("nan")
    names = list(want)
    outs = {n: torch.full(tuple(want[n].shape), 7.0, device="cuda",
                          dtype=torch.float32 if n in ("dlog_decay", "dh0") else IO[io]) for n in names}
    agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=starts(spans) if packed else None,
                     h0=t["h0"], dhT=t["dhT"], scale=scale, grads=outs)
    torch.cuda.synchronize()
    for n in names:
        got, w = outs[n].cpu(), want[n]
        if n != "dh0" and not (n == "dlog_decay" and d["g"].dim() == 1):
            assert bool((got[out] == 7.0).all()), n
            got, w = got[~out], w[~out]
        check(n, got, w, io, "gradient")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_gradient_subsets_agree(agm, io):
    """Any choice of outputs gives what the whole set gives (dq, dk and dv do
    not need the decay's gradient: without it their state operands are
    rounded once, which is within the same tolerance)."""
    c = dict(lens=[300, 90], Hk=1, Hv=2, dk=64, dv=64, states=True)
    spans, T, d, scale = build(c, io, 13)
    want, _ = ref.gradient(d["q"], d["k"], d["v"], d["g"], d["dy"], spans, scale, d["h0"], d["dhT"])
    t = device_inputs(d, io)
    for names in (["dq"], ["dk"], ["dv"], ["dlog_decay"], ["dh0"], ["dq", "dk", "dv"], ["dv", "dh0"], ["dk", "dh0"]):
        got = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=starts(spans), h0=t["h0"],
                               dhT=t["dhT"], scale=scale, want=names)
        assert list(got) == names
        for n in names:
            check(n, got[n].cpu(), want[n], io, "+".join(names))


def test_gradient_against_differences(agm):
    c = dict(lens=[70, 9], Hk=1, Hv=2, dk=16, dv=8, states=True)
    spans, T, d, scale = build(c, "f32", 14)
    t = device_inputs(d, "f32")
    got = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=starts(spans), h0=t["h0"], dhT=t["dhT"],
                           scale=scale)
    rng = torch.Generator().manual_seed(5)
    for n, x in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dlog_decay", "g"), ("dh0", "h0")):
        step = torch.randn(d[x].shape, generator=rng, dtype=torch.float64)
        eps = 1e-6
        ls = []
        for sign in (1, -1):
            e = dict(d)
            e[x] = d[x] + sign * eps * step
            y, hT = ref.forward(e["q"], e["k"], e["v"], e["g"], spans, scale, e["h0"])
            ls.append(float((d["dy"] * y).sum() + (d["dhT"] * hT).sum()))
        want = (ls[0] - ls[1]) / (2 * eps)
        have = float((got[n].double().cpu() * step).sum())
        # second-order differences leave eps^2, the sums of fp64 losses 1e-16 / eps; fp32 gradients 2^-18
        size = float((got[n].double().cpu().abs() * step.abs()).sum())
        assert abs(have - want) <= 2.0 ** -18 * size, (n, have, want)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strong_and_missing_decays(agm, io):
    """Resets (-inf), decays that underflow, none at all, and a growing head."""
    c = dict(lens=[150, 64], Hk=1, Hv=4, dk=32, dv=32, states=True)
    spans, T, d, scale = build(c, io, 15)
    g = d["g"]
    g[:, 0] = 0.0
    g[::7, 1] = float("-inf")
    g[:, 2] = -90.0
    g[::13, 2] = -1e30
    g[:, 3] = 0.01
    want, ends = ref.forward(d["q"], d["k"], d["v"], g, spans, scale, d["h0"])
    gw, _ = ref.gradient(d["q"], d["k"], d["v"], g, d["dy"], spans, scale, d["h0"], d["dhT"])
    # d exp(g) / dg at -inf: autograd forms 0 * (finite) = 0
    t = device_inputs(d, io)
    y, hT = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=starts(spans), h0=t["h0"], scale=scale,
                                want_state=True)
    got = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=starts(spans), h0=t["h0"], dhT=t["dhT"],
                           scale=scale)
    for h in range(4):
        check(f"y head {h}", y[:, h].cpu(), want[:, h], io, "decays")
        check(f"hT head {h}", hT[:, h].cpu(), ends[:, h], io, "decays")
        check(f"dv head {h}", got["dv"][:, h].cpu(), gw["dv"][:, h], io, "decays")
        if h != 2:
            check(f"dg head {h}", got["dlog_decay"][:, h].cpu(), gw["dlog_decay"][:, h], io, "decays")
        else:  # e^-90 of anything here is zero in fp32
            assert float(got["dlog_decay"][:, h].abs().max()) <= 1e-30
    for n in ("dq", "dk", "dh0"):
        check(n, got[n].cpu(), gw[n], io, "decays")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_strided_rows(agm, io):
    """q, k, v as slices of one projection's rows, y and dy as slices too: the
    same bits as contiguous copies."""
    T, H, dk, dv = 333, 2, 64, 32
    d = ref.inputs(16, T, H, H, dk, dv, io)
    t = device_inputs(d, io)
    rows = torch.cat([t["q"].flatten(1), t["k"].flatten(1), t["v"].flatten(1)], dim=1)
    q, k, v = rows[:, :128].unflatten(1, (H, dk)), rows[:, 128:256].unflatten(1, (H, dk)), rows[:, 256:].unflatten(1, (H, dv))
    wide = torch.zeros(T, 2 * H * dv, dtype=IO[io], device="cuda")
    yv = wide[:, H * dv:].unflatten(1, (H, dv))
    a, _ = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"])
    agm.linattn_forward(q, k, v, t["g"], y=yv)
    assert torch.equal(a, yv) and not bool(wide[:, :H * dv].any())
    wide[:, H * dv:] = t["dy"].flatten(1)
    g0 = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"])
    g1 = agm.linattn_grad(q, k, v, t["g"], yv)
    for n in g0:
        assert torch.equal(g0[n], g1[n]), n
    st0 = torch.ones(T, H, dk, dv, device="cuda")
    st1 = st0.clone()
    assert torch.equal(agm.linattn_step(t["q"], t["k"], t["v"], t["g"], st0), agm.linattn_step(q, k, v, t["g"], st1))
    assert torch.equal(st0, st1)


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_batch_of_equal_sequences(agm, io):
    """[S, L, H, d] is the packed call with equal lengths."""
    S, L, H, dk, dv = 3, 130, 2, 64, 64
    d = ref.inputs(17, S * L, H, H, dk, dv, io, S=S, states=True)
    t = device_inputs(d, io)
    spans = spans_of([L] * S)
    y0, h0 = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=starts(spans), h0=t["h0"], want_state=True)
    b = {n: t[n].unflatten(0, (S, L)) for n in ("q", "k", "v", "g", "dy")}
    y1, h1 = agm.linattn_forward(b["q"], b["k"], b["v"], b["g"], h0=t["h0"], want_state=True)
    assert torch.equal(y0, y1.flatten(0, 1)) and torch.equal(h0, h1)
    g0 = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=starts(spans), h0=t["h0"], dhT=t["dhT"])
    g1 = agm.linattn_grad(b["q"], b["k"], b["v"], b["g"], b["dy"], h0=t["h0"], dhT=t["dhT"])
    for n in g0:
        assert torch.equal(g0[n].flatten(), g1[n].flatten()), n


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hk,Hv,dk,dv,decay", [(1, 1, 1, 8, 8, "token"), (3, 2, 4, 128, 128, "head"),
                                                 (7, 1, 3, 40, 104, "token"), (300, 1, 2, 64, 64, "token")])
def test_step(agm, io, B, Hk, Hv, dk, dv, decay):
    d = ref.inputs(18, B, Hk, Hv, dk, dv, io, decay, B, True)
    if decay == "token":
        d["g"][0, 0] = float("-inf")
    spans = [(t, t + 1) for t in range(B)]
    want, ends = ref.forward(d["q"], d["k"], d["v"], d["g"], spans, 0.3, d["h0"])
    t = device_inputs(d, io)
    st = t["h0"].clone()
    y = agm.linattn_step(t["q"], t["k"], t["v"], t["g"], st, scale=0.3)
    # fp32 inside for both types: one rounding of y, a few of the state
    check("y", y.cpu(), want, io, "step")
    assert ref.rms_err(st, ends) <= 2.0 ** -22


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_prompt_then_steps(agm, io):
    """A prompt's final states continued token by token give the outputs of
    the whole sequences."""
    H, dk, dv, n, more = 2, 64, 64, [100, 37, 0], 5
    spans = spans_of([c + more for c in n])
    T = spans[-1][1]
    d = ref.inputs(19, T, H, H, dk, dv, io)
    want, ends = ref.forward(d["q"], d["k"], d["v"], d["g"], spans, 1.0)
    t = device_inputs(d, io)
    idx = torch.cat([torch.arange(a, a + c) for (a, _), c in zip(spans, n)]).cuda()
    ps = spans_of(n)
    y, st = agm.linattn_forward(t["q"][idx], t["k"][idx], t["v"][idx], t["g"][idx], seq_start=starts(ps),
                                want_state=True)
    check("prompt y", y.cpu(), want[idx.cpu()], io, "serve")
    for s in range(more):
        row = torch.tensor([a + c + s for (a, _), c in zip(spans, n)])
        r = row.cuda()
        y = agm.linattn_step(t["q"][r], t["k"][r], t["v"][r], t["g"][r], st)
        check(f"step {s} y", y.cpu(), want[row], io, "serve")
    check("states", st.cpu(), ends, io, "serve")


def test_state_in_place_and_on_another_stream(agm):
    d = ref.inputs(20, 600, 1, 2, 64, 64, "bf16", S=1, states=True)
    t = device_inputs(d, "bf16")
    y0, h0 = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], want_state=True)
    h = t["h0"].clone()
    y1, h1 = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], h0=h, hT=h)
    assert h1 is h and torch.equal(y0, y1) and torch.equal(h0, h)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    y2, h2 = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], want_state=True, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y0, y2) and torch.equal(h0, h2)


def test_captured_and_replayed(agm):
    """A captured prompt, gradient and step, replayed with other inputs and
    other sequence lengths, give the eager results; two graphs with
    workspaces of their own do not disturb each other."""
    T, H, dk, dv, S = 700, 2, 64, 64, 3
    lens = [[700, 0, 0], [1, 300, 200], [64, 64, 500]]
    ins = [device_inputs(ref.inputs(30 + i, T, H, H, dk, dv, "bf16", S=S, states=True), "bf16") for i in range(3)]
    st = {n: x.clone() for n, x in ins[0].items()}
    off = starts(spans_of(lens[0]))

    def work():
        y, hT = agm.linattn_forward(st["q"], st["k"], st["v"], st["g"], seq_start=off, h0=st["h0"], want_state=True)
        g = agm.linattn_grad(st["q"], st["k"], st["v"], st["g"], st["dy"], seq_start=off, h0=st["h0"], dhT=st["dhT"])
        ys = agm.linattn_step(st["q"][:S], st["k"][:S], st["v"][:S], st["g"][:S], hT)
        return [y, hT, ys] + [g[n] for n in agm.linattn.GRADS]

    work()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(work())
        graphs.append(g)
    for i in (1, 2, 0, 1):
        for n in st:
            st[n].copy_(ins[i][n])
        off.copy_(starts(spans_of(lens[i])))
        for o in outs:
            for x in o:
                x.zero_()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        used = sum(lens[i])
        want = work()
        for o in outs:
            for j, (a, b) in enumerate(zip(o, want)):
                rows = a.shape[0] if a.shape[0] != T else used
                assert torch.equal(a[:rows], b[:rows]), (i, j)


def test_bad_offsets_stay_inside(agm):
    """Offsets out of order or out of range give no access outside the
    arrays: rows of the guard buffers around every output keep their value."""
    T, H, d = 256, 1, 64
    x = ref.inputs(40, T, H, H, d, d, "bf16", S=4, states=True)
    t = device_inputs(x, "bf16")
    for bad in ([0, 500, 20, 256, 100], [-5, 10, 3, 1 << 30, 40], [200, 100, 50, 20, 0]):
        off = torch.tensor(bad, dtype=torch.int32, device="cuda")
        buf = torch.full((T + 128, H, d), 3.0, dtype=torch.bfloat16, device="cuda")
        agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=off, h0=t["h0"], y=buf[64:64 + T])
        agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=off, h0=t["h0"], dhT=t["dhT"])
        torch.cuda.synchronize()
        assert bool((buf[:64] == 3.0).all()) and bool((buf[64 + T:] == 3.0).all())


def test_repeatable(agm):
    d = ref.inputs(41, 900, 1, 3, 128, 64, "bf16", "head", 2, True)
    t = device_inputs(d, "bf16")
    off = starts(spans_of([500, 400]))
    runs = [agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=off, h0=t["h0"], dhT=t["dhT"])
            for _ in range(3)]
    for r in runs[1:]:
        for n in r:
            assert torch.equal(r[n], runs[0][n]), n
