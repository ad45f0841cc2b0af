"""The operators at their edges on the GPU: many and long sequences, offsets
past 32 bits, non-finite tokens, streams, refusals of GPU tensors."""
import pytest
import torch

import linattn_ref as ref
from gpu_util import say
from test_gpu_linattn import IO, check, device_inputs, spans_of, starts

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def agm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import adjoint_gradients_amd as agm

    return agm


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_many_sequences(agm, io):
    """More sequences than any table or wavefront holds, most of them short or empty."""
    gen = torch.Generator().manual_seed(7)
    lens = [int(x) for x in torch.randint(0, 9, (150,), generator=gen)] + [0, 301, 0, 65, 1]
    spans = spans_of(lens, 2)
    T = spans[-1][1] + 1
    d = ref.inputs(50, T, 1, 2, 24, 16, io, S=len(lens), states=True)
    want, ends = ref.forward(d["q"], d["k"], d["v"], d["g"], spans, 0.5, d["h0"])
    gw, _ = ref.gradient(d["q"], d["k"], d["v"], d["g"], d["dy"], spans, 0.5, d["h0"], d["dhT"])
    t = device_inputs(d, io)
    off = starts(spans)
    y, hT = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=off, h0=t["h0"], scale=0.5, want_state=True)
    got = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=off, h0=t["h0"], dhT=t["dhT"], scale=0.5)
    check("y", y[2:T - 1].cpu(), want[2:T - 1], io, "many")
    check("hT", hT.cpu(), ends, io, "many")
    for n in got:
        rows = slice(None) if n == "dh0" else slice(2, T - 1)
        check(n, got[n].cpu()[rows], gw[n][rows], io, "many")


def test_offsets_past_32_bits(agm):
    """v, y and their cotangents of 2.2e9 elements: the last head against the
    same head computed alone (other segments, so other fp32 carries)."""
    T, Hv, dk, dv = 133000, 130, 16, 128
    assert T * Hv * dv > 2 ** 31
    gen = torch.Generator(device="cuda").manual_seed(3)
    q = torch.randn(T, 1, dk, generator=gen, device="cuda").bfloat16()
    k = torch.randn(T, 1, dk, generator=gen, device="cuda").bfloat16()
    v = torch.empty(T, Hv, dv, dtype=torch.bfloat16, device="cuda")
    dy = torch.empty_like(v)
    v.normal_(generator=gen)
    dy.normal_(generator=gen)
    g = -torch.rand(T, Hv, generator=gen, device="cuda") * 0.1
    say("case forward")
    y, hT = agm.linattn_forward(q, k, v, g, want_state=True)
    h = Hv - 1
    one = [v[:, h:].contiguous(), g[:, h:].contiguous(), dy[:, h:].contiguous()]
    y1, h1 = agm.linattn_forward(q, k, one[0], one[1], want_state=True)
    # one output rounding each, and the fp32 sums before it
    assert ref.rms_err(y[:, h:], y1.double().cpu()) <= 2.0 ** -8
    assert ref.rms_err(hT[:, h:], h1.double().cpu()) <= 2.0 ** -18
    say("case gradient")
    a = agm.linattn_grad(q, k, v, g, dy, want=["dv", "dlog_decay"])
    b = agm.linattn_grad(q, k, one[0], one[1], one[2], want=["dv", "dlog_decay"])
    assert ref.rms_err(a["dv"][:, h:], b["dv"].double().cpu()) <= 2.0 ** -8
    assert ref.rms_err(a["dlog_decay"][:, h:], b["dlog_decay"].double().cpu()) <= 2.0 ** -16


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_nonfinite_tokens_stay_in_their_sequence_and_head(agm, io):
    spans = spans_of([100, 70, 300])
    T = spans[-1][1]
    d = ref.inputs(51, T, 2, 2, 32, 32, io, S=3, states=True)
    t = device_inputs(d, io)
    clean = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=starts(spans), h0=t["h0"], want_state=True)
    gclean = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=starts(spans), h0=t["h0"], dhT=t["dhT"])
    for n, bad in (("v", float("inf")), ("k", float("nan")), ("dy", float("nan"))):
        u = {m: (None if x is None else x.clone()) for m, x in t.items()}
        u[n][130, 0] = bad  # a token of the second sequence, first head
        y, hT = agm.linattn_forward(u["q"], u["k"], u["v"], u["g"], seq_start=starts(spans), h0=u["h0"], want_state=True)
        got = agm.linattn_grad(u["q"], u["k"], u["v"], u["g"], u["dy"], seq_start=starts(spans), h0=u["h0"], dhT=u["dhT"])
        out = torch.ones(T, dtype=torch.bool, device="cuda")
        out[100:170] = False
        assert torch.equal(y[out], clean[0][out]) and torch.equal(y[:, 1], clean[0][:, 1])
        assert torch.equal(hT[[0, 2]], clean[1][[0, 2]]) and torch.equal(hT[:, 1], clean[1][:, 1])
        for m in ("dq", "dk", "dv", "dlog_decay"):
            assert torch.equal(got[m][out], gclean[m][out]) and torch.equal(got[m][:, 1], gclean[m][:, 1]), (n, m)


def test_two_streams_at_once(agm):
    """Calls on two streams with their own workspaces and inputs, interleaved."""
    ins = [device_inputs(ref.inputs(60 + i, 1500, 2, 2, 64, 64, "bf16", S=1, states=True), "bf16") for i in range(2)]

    def work(t):
        y, hT = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], h0=t["h0"], want_state=True)
        g = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], h0=t["h0"], dhT=t["dhT"])
        x, r, ri = agm.add_norm(t["h0"].view(-1, 64), None, t["h0"].view(-1)[:64].contiguous(), io="bf16")
        n = agm.clip_grads([g["dlog_decay"], g["dh0"]], 0.5)
        return [y, hT, g["dq"], g["dk"], g["dv"], g["dlog_decay"], g["dh0"], x, ri, n]

    want = [work(t) for t in ins]
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in ins]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(side):
            with torch.cuda.stream(s):
                got[i].append(work(ins[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for run in got[i]:
            for a, b in zip(run, want[i]):
                assert torch.equal(a, b)


def test_an_explicit_stream_owns_what_the_call_makes(agm):
    s = torch.cuda.Stream()
    t = device_inputs(ref.inputs(62, 700, 1, 1, 64, 64, "bf16"), "bf16")
    want = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"])
    r, dx = t["g"].expand(700, 64).contiguous(), t["dy"].view(700, 64)
    gm = torch.ones(64, device="cuda")
    wn = agm.add_norm(r, dx, gm)
    wg = agm.add_norm_grad(wn[1], wn[2], gm, dx)
    torch.cuda.synchronize()
    for _ in range(3):
        g = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], stream=s.cuda_stream)
        n = agm.add_norm(r, dx, gm, stream=s.cuda_stream)
        s.synchronize()
        gg = agm.add_norm_grad(n[1], n[2], gm, dx, stream=s.cuda_stream)
        norm = agm.clip_grads([gg[0]], float("inf"), stream=s.cuda_stream)
        s.synchronize()
        assert all(torch.equal(g[m], want[m]) for m in want)
        assert all(torch.equal(a, b) for a, b in zip(n, wn)) and all(torch.equal(a, b) for a, b in zip(gg, wg))
        assert abs(float(norm) - float(wg[0].double().norm())) <= 1e-6 * float(norm)


def test_refusals_of_gpu_tensors(agm):
    q = torch.zeros(6, 2, 16, device="cuda", dtype=torch.bfloat16)
    v = torch.zeros(6, 4, 8, device="cuda", dtype=torch.bfloat16)
    g = torch.zeros(6, 4, device="cuda")
    ok = lambda **kw: agm.linattn_forward(**{**dict(q=q, k=q, v=v, log_decay=g), **kw})
    ok()
    off = lambda *x, dtype=torch.int32: torch.tensor(x, dtype=dtype, device="cuda")
    for kw, word in ((dict(k=q[:5]), "shape"), (dict(k=q.float()), "dtype"), (dict(v=v[:, :, ::2]), "contiguous"),
                     (dict(log_decay=g.double()), "dtype"), (dict(log_decay=g[:, :3]), "shape"),
                     (dict(log_decay=torch.zeros(3, device="cuda")), "shape"),
                     (dict(h0=torch.zeros(1, 4, 16, 9, device="cuda")), "shape"),
                     (dict(seq_start=off(0, 6, dtype=torch.int64)), "dtype"), (dict(seq_start=off(0)), "offsets"),
                     (dict(y=torch.zeros(6, 4, 8, device="cuda")), "dtype"), (dict(k=q.cpu()), "GPU tensor"),
                     (dict(ws=torch.zeros(4, device="cuda")), "dtype"), (dict(q=q.half(), k=q.half()), "dtype")):
        with pytest.raises(agm.SsmError, match=word):
            ok(**kw)
    with pytest.raises(agm.SsmError, match="UNSUPPORTED"):
        agm.linattn_forward(q[:, :, :12].contiguous(), q[:, :, :12].contiguous(), v, g)
    with pytest.raises(agm.SsmError, match="ERR_ARG"):  # two value heads for three key heads
        agm.linattn_forward(torch.zeros(6, 3, 16, device="cuda"), torch.zeros(6, 3, 16, device="cuda"),
                            torch.zeros(6, 4, 8, device="cuda"), g)
    with pytest.raises(agm.SsmError, match="none of"):
        agm.linattn_grad(q, q, v, g, v, want=["dx"])
    with pytest.raises(agm.SsmError):
        agm.linattn_grad(q, q, v, g, v, want=[])
    with pytest.raises(agm.SsmError, match="shape"):
        agm.linattn_step(q, q, v, g, torch.zeros(5, 4, 16, 8, device="cuda"))
    with pytest.raises(agm.SsmError, match="dimensions"):
        agm.linattn_step(q[None], q[None], v[None], g[None], torch.zeros(6, 4, 16, 8, device="cuda"))
    r = torch.zeros(4, 8, device="cuda")
    for call, word in ((lambda: agm.add_norm(r, r.bfloat16()[:3], torch.ones(8, device="cuda")), "shape"),
                       (lambda: agm.add_norm(r, r.half(), torch.ones(8, device="cuda")), "io dtype"),
                       (lambda: agm.add_norm(r, None, torch.ones(7, device="cuda"), io="f32"), "shape"),
                       (lambda: agm.add_norm(r, None, torch.ones(8, device="cuda")), "io dtype"),
                       (lambda: agm.add_norm(r.t(), None, torch.ones(4, device="cuda"), io="f32"), "contiguous"),
                       (lambda: agm.add_norm_grad(r, torch.ones(3, device="cuda"), torch.ones(8, device="cuda"), r), "shape"),
                       (lambda: agm.clip_grads([r, r], 1.0), "twice"),
                       (lambda: agm.clip_grads([r, r.bfloat16()], 1.0), "dtype"),
                       (lambda: agm.clip_grads([r], 0.0), "positive"),
                       (lambda: agm.clip_grads([r], 1.0, out=[r[:2]]), "shape"),
                       (lambda: agm.clip_grads([r], 1.0, out=[]), "outputs"),
                       (lambda: agm.clip_grads([r.t()], 1.0), "contiguous")):
        with pytest.raises(agm.SsmError, match=word):
            call()


def test_clip_outputs_that_meet(agm):
    """One output for two gradients, and an output that is another gradient: refused, nothing written."""
    a, b, c = (torch.full((40,), float(i + 1), device="cuda") for i in range(3))
    none = torch.empty(0, device="cuda")
    for ts, out in (([a, b], [c, c]), ([a, b], [b, c]), ([a, a], [a, c])):
        with pytest.raises(agm.SsmError):
            agm.clip_grads(ts, 1.0, out=out)
    assert [float(t.sum()) for t in (a, b, c)] == [40.0, 80.0, 120.0]
    # in place beside a separate output, the same input twice, empty tensors at one address
    n = agm.clip_grads([a, b, none, none], 1.0, out=[a, c, none, none])
    assert abs(float(n) - (40 * 1 + 40 * 4) ** 0.5) < 1e-4
    d, e = torch.empty_like(b), torch.empty_like(b)
    agm.clip_grads([b, b], 1e9, out=[d, e])
    assert torch.equal(d, b) and torch.equal(e, b)


@pytest.mark.parametrize("lens,Hk,Hv,dk,dv,states", [
    ([1], 2, 4, 64, 64, False), ([1, 1], 3, 3, 8, 104, True), ([5, 2], 1, 6, 40, 24, True),
    ([19], 2, 2, 128, 128, False), ([130, 64], 1, 2, 72, 128, True)])
def test_bf16_rounded_once(agm, lens, Hk, Hv, dk, dv, states):
    """Every bf16 output is off by its own rounding, half a step (2^-8 of it at
    most), and by 2^-15 of the sum's absolute values: two operands in two bf16
    parts each, 2^-17 apiece, and the fp32 sums (under 2^-16 for these lengths)."""
    spans = spans_of(lens, 0)
    T = spans[-1][1]
    d = ref.inputs(60, T, Hk, Hv, dk, dv, "bf16", S=len(lens), states=states)
    mag = {n: (x if n == "g" or x is None else x.abs()) for n, x in d.items()}
    t = device_inputs(d, "bf16")
    off = starts(spans)
    y, _ = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=off, h0=t["h0"], scale=0.3)
    got = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=off, h0=t["h0"], dhT=t["dhT"], scale=0.3)
    plain = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=off, h0=t["h0"], dhT=t["dhT"], scale=0.3,
                             want=["dq", "dk", "dv"])
    refs = []
    for x in (d, mag):
        r, _ = ref.gradient(x["q"], x["k"], x["v"], x["g"], x["dy"], spans, 0.3, x["h0"], x["dhT"])
        refs.append({"y": ref.forward(x["q"], x["k"], x["v"], x["g"], spans, 0.3, x["h0"])[0], **r})
    for n, out in (("y", [y]), ("dq", [got["dq"], plain["dq"]]), ("dk", [got["dk"], plain["dk"]]),
                   ("dv", [got["dv"], plain["dv"]])):
        for o in out:
            over = (o.double().cpu() - refs[0][n]).abs() - 2.0 ** -8 * refs[0][n].abs() - 2.0 ** -15 * refs[1][n]
            assert float(over.max()) <= 0, (n, float(over.max()))


@pytest.mark.parametrize("io,lens,Hk,Hv,dk,dv", [
    ("f32", [1700], 1, 1, 8, 24), ("f32", [1030, 0, 131, 1, 64], 2, 2, 40, 16), ("bf16", [2300], 1, 2, 64, 32)])
def test_long_walks_of_few_states(agm, io, lens, Hk, Hv, dk, dv):
    """More segments than parts of a carried walk, not a multiple of them, beside
    sequences of one segment and none; decays slow enough to reach across them."""
    spans = spans_of(lens, 0)
    T = spans[-1][1]
    d = ref.inputs(61, T, Hk, Hv, dk, dv, io, S=len(lens), states=True)
    d["g"] = d["g"] * 0.05
    want, ends = ref.forward(d["q"], d["k"], d["v"], d["g"], spans, 0.5, d["h0"])
    gw, _ = ref.gradient(d["q"], d["k"], d["v"], d["g"], d["dy"], spans, 0.5, d["h0"], d["dhT"])
    t = device_inputs(d, io)
    off = starts(spans)
    y, hT = agm.linattn_forward(t["q"], t["k"], t["v"], t["g"], seq_start=off, h0=t["h0"], scale=0.5, want_state=True)
    got = agm.linattn_grad(t["q"], t["k"], t["v"], t["g"], t["dy"], seq_start=off, h0=t["h0"], dhT=t["dhT"], scale=0.5)
    check("y", y.cpu(), want, io, "walks")
    check("hT", hT.cpu(), ends, io, "walks")
    for n in got:
        check(n, got[n].cpu(), gw[n], io, "walks")


@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_step_of_many_states(agm, io):
    """States larger than the caches keep, in widths that fill no tile; a second step finds the first one's."""
    B, Hk, Hv, dk, dv = 43, 8, 32, 120, 104
    d = ref.inputs(62, B, Hk, Hv, dk, dv, io, S=B, states=True)
    t = device_inputs(d, io)
    q, k = (d[n].repeat_interleave(Hv // Hk, dim=1) for n in ("q", "k"))
    st, h = t["h0"].clone(), d["h0"]
    for _ in range(2):
        h = torch.exp(d["g"])[..., None, None] * h + k[..., None] * d["v"][:, :, None, :]
        y = agm.linattn_step(t["q"], t["k"], t["v"], t["g"], st, scale=0.5)
        check("y", y.cpu(), 0.5 * (q[..., None] * h).sum(2), io, "many states")
    assert ref.rms_err(st.cpu(), h) <= 2.0 ** -22  # two steps of two fp32 roundings each


@pytest.mark.parametrize("io,n", [("f32", 51_000_003), ("bf16", 101_000_005)])
def test_clip_more_than_the_caches(agm, io, n):
    """Gradients that the caches do not hold, into other tensors and in place: every element is the
    input times one factor, rounded once (half a step), the factor off by 2^-23 (its own rounding and the norm's)."""
    t = torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(9)).to(IO[io])
    ts = [t[: n // 3].clone(), t[n // 3: n // 3].clone(), t[n // 3:].clone()]
    total = float(sum(x.double().square().sum() for x in ts)) ** 0.5
    out = [torch.empty_like(x) for x in ts]
    norm = agm.clip_grads(ts, total / 3, out=out)
    assert abs(float(norm) - total) <= 2.0 ** -23 * total
    again = [x.clone() for x in ts]
    agm.clip_grads(again, total / 3)
    tol = torch.finfo(IO[io]).eps / 2 + 2.0 ** -23
    for x, o, a in zip(ts, out, again):
        assert torch.equal(o, a)
        want = x.double() / 3
        assert bool(((o.double() - want).abs() <= tol * want.abs()).all())
