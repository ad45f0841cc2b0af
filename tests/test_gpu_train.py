"""The residual update with its norm, and gradient clipping, against 64 bits.

Roundings: fp32 results are a few roundings off, 2^-24 each, plus those of a
sum of P or T squares (about sqrt(n) 2^-24): 2^-20 in the mean square covers
16.  bf16 results add their own rounding, 2^-8 / sqrt(3) in the mean square."""
import math

import pytest
import torch

from gpu_util import say

pytestmark = pytest.mark.gpu

IO = {"bf16": torch.bfloat16, "f32": torch.float32}
TOL = {torch.float32: 2.0 ** -20, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def agm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import adjoint_gradients_amd as agm

    return agm


def check(name, got, want, size=None):
    """size: the terms whose difference the result is, when they can cancel."""
    d = float((got.double() - want).square().mean().sqrt())
    n = float((want if size is None else size).square().mean().sqrt())
    err = d / n if n else d
    say(f"  {name}: rms error {err:.2e} (<= {TOL[got.dtype]:.2e})")
    assert err <= TOL[got.dtype], (name, err)


def randn(gen, *shape, dtype=torch.float32, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# one row, rows of each kernel shape, odd widths, the widest
SIZES = [(1, 1), (3, 17), (5, 2048), (2500, 512), (2500, 300), (2050, 1999), (4100, 1536), (3, 2052), (9, 8191),
         (2, 8196), (2, 16384), (1, 16383)]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("T,P", SIZES)
def test_add_norm_and_gradient(agm, T, P, io):
    g = gen_of(T * 31 + P)
    r, y = randn(g, T, P, scale=2.0), randn(g, T, P, dtype=IO[io])
    gm = 1.0 + randn(g, P, scale=0.2)
    x, ro, ri = agm.add_norm(r, y, gm, eps=1e-5)
    r64 = r.double() + y.double()
    ri64 = (r64.square().mean(1) + 1e-5).rsqrt()
    check("r_out", ro, r64)
    check("rinv", ri, ri64)
    check("x", x, gm.double() * r64 * ri64[:, None])
    dx, do = randn(g, T, P, dtype=IO[io]), randn(g, T, P)
    dr, ds = agm.add_norm_grad(ro, ri, gm, dx, do)
    xh = ro.double() * ri.double()[:, None]
    u = gm.double() * dx.double()
    want = do.double() + ri.double()[:, None] * (u - xh * (u * xh).mean(1, keepdim=True))
    check("dr", dr, want)
    check("dnorm_scale", ds, (dx.double() * xh).sum(0))
    # the same in place, without y, without dr_out
    do2 = do.clone()
    dr2, none = agm.add_norm_grad(ro, ri, gm, dx, do2, dr=do2, want_scale=False)
    assert dr2 is do2 and none is None and torch.equal(dr2, dr)
    r2 = r.clone()
    x2, ro2, _ = agm.add_norm(r2, y, gm, r_out=r2)
    assert ro2 is r2 and torch.equal(r2, ro) and torch.equal(x2, x)
    x3, ro3, ri3 = agm.add_norm(ro, None, gm, io=io)
    assert ro3 is ro and torch.equal(x3, x) and torch.equal(ri3, ri)
    dr4, _ = agm.add_norm_grad(ro, ri, gm, dx)
    # rinv (u - xh m): for P = 1 xh is +-1 up to eps and u - xh m cancels all
    # but the part eps leaves (here 5e-6 of u), so the roundings of the two
    # terms, 2^-24 each, count against rinv u
    check("dr without dr_out", dr4, want - do.double(), ri.double()[:, None] * u)


def test_norm_gradient_against_differences(agm):
    g = gen_of(3)
    T, P = 4, 24
    r, y, gm = randn(g, T, P), randn(g, T, P), 1.0 + randn(g, P, scale=0.2)
    dx, do = randn(g, T, P), randn(g, T, P)
    x, ro, ri = agm.add_norm(r, y, gm)
    dr, ds = agm.add_norm_grad(ro, ri, gm, dx, do)

    def loss(r, gm):
        s = r + y.double()
        return float((dx.double() * gm * s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt()).sum()
                     + (do.double() * s).sum())

    step, eps = randn(g, T, P).double(), 1e-6
    want = (loss(r.double() + eps * step, gm.double()) - loss(r.double() - eps * step, gm.double())) / (2 * eps)
    assert abs(float((dr.double() * step).sum()) - want) <= 2.0 ** -18 * float((dr.double() * step).abs().sum())
    step = randn(g, P).double()
    want = (loss(r.double(), gm.double() + eps * step) - loss(r.double(), gm.double() - eps * step)) / (2 * eps)
    assert abs(float((ds.double() * step).sum()) - want) <= 2.0 ** -18 * float((ds.double() * step).abs().sum())


def test_norm_of_zero_rows_and_nonfinite_rows(agm):
    r = torch.zeros(3, 64, device="cuda")
    r[1, 5] = float("inf")
    r[2] = 1.0
    y = torch.zeros(3, 64, device="cuda", dtype=torch.bfloat16)
    x, ro, ri = agm.add_norm(r, y, torch.ones(64, device="cuda"), eps=1e-5)
    assert not bool(x[0].any()) and abs(float(ri[0]) - 1e-5 ** -0.5) < 1e-3 * 1e-5 ** -0.5
    # a row's infinity stays in its row
    assert bool(torch.isfinite(x[2].float()).all()) and float(x[2, 0]) == 1.0


SETS = [[(1,)], [(64, 64), (16, 64), (64, 16), (64,)], [(8192,), (8193,), (8191,), (0,), (3, 5)],
        [(7,)] * 300, [(1000, 1001), (0, 4), (2048, 2048)]]


@pytest.mark.parametrize("io", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(SETS)))
def test_clip(agm, i, io):
    g = gen_of(50 + i)
    ts = [randn(g, *s, dtype=IO[io]) for s in SETS[i]]
    total = math.sqrt(math.fsum(float(t.double().square().sum()) for t in ts))
    before = [t.clone() for t in ts]
    out = [torch.empty_like(t) for t in ts]
    # out of place, in place, above the norm, and the norm alone
    for max_norm in (total / 3, total * 2):
        c = max_norm / total if total > max_norm else 1.0
        n = agm.clip_grads(ts, max_norm, out=out)
        assert abs(float(n) - total) <= 2.0 ** -23 * total
        for t, o, b in zip(ts, out, before):
            assert torch.equal(t, b)
            if c == 1.0:
                assert torch.equal(o, b)
            elif t.numel():
                # the coefficient's rounding, the product's, and the io type's own
                half = torch.finfo(IO[io]).eps / 2
                assert bool(((o.double() - b.double() * c).abs() <= (half + 2.0 ** -23) * (b.double() * c).abs()).all())
    n = agm.clip_grads(ts, float("inf"))
    assert abs(float(n) - total) <= 2.0 ** -23 * total and all(torch.equal(t, b) for t, b in zip(ts, before))
    agm.clip_grads(ts, total / 3, out=out)
    agm.clip_grads(ts, total / 3)
    assert all(torch.equal(t, o) for t, o in zip(ts, out))


def test_clip_range_and_nonfinite(agm):
    # squares that overflow or vanish in fp32
    for scale in (1e25, 1e-30):
        t = torch.full((1000,), scale, device="cuda")
        n = agm.clip_grads([t], scale)
        want = scale * math.sqrt(1000)
        assert abs(float(n) - want) <= 1e-6 * want
        assert bool(((t.double() / (scale / math.sqrt(1000)) - 1).abs() <= 1e-6).all())
    for bad in (float("nan"), float("inf"), float("-inf")):
        t = torch.ones(100, device="cuda")
        t[7] = bad
        b = t.clone()
        n = agm.clip_grads([t, torch.ones(5, device="cuda")], 0.5)
        assert not math.isfinite(float(n)) and torch.equal(t.nan_to_num(9.0), b.nan_to_num(9.0))


def test_capture(agm):
    g = gen_of(70)
    T, P = 300, 256
    r, y, gm = randn(g, T, P), randn(g, T, P, dtype=torch.bfloat16), 1.0 + randn(g, P, scale=0.2)
    dx, do = randn(g, T, P, dtype=torch.bfloat16), randn(g, T, P)

    def work():
        x, ro, ri = agm.add_norm(r, y, gm)
        dr, ds = agm.add_norm_grad(ro, ri, gm, dx, do)
        n = agm.clip_grads([ds, dr], 1.0)
        return [x, ro, ri, dr, ds, n]

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(3):
        for t in (r, do):
            t.copy_(randn(g, T, P))
        y.copy_(randn(g, T, P))
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, work()):
            assert torch.equal(a, b)


def test_a_training_step_together(agm):
    """Norm, attention, loss cotangent, their gradients, clipping: the
    gradients of a residual block against autograd in 64 bits, then their norm."""
    g = gen_of(80)
    T, H, d = 130, 2, 32
    P = H * d
    r, gm = randn(g, T, P), 1.0 + randn(g, P, scale=0.2)
    y0 = randn(g, T, P)
    lg = -torch.rand(T, H, generator=g, device="cuda") * 0.2
    do = randn(g, T, P)
    # block: x = norm(r + y0); r2 = r + y0 + attention(x, x, x)
    x, ro, ri = agm.add_norm(r, y0, gm)
    h = x.view(T, H, d)
    y, _ = agm.linattn_forward(h, h, h, lg, scale=0.1)
    gr = agm.linattn_grad(h, h, h, lg, do.view(T, H, d), scale=0.1)
    dx = gr["dq"] + gr["dk"] + gr["dv"]
    dr, ds = agm.add_norm_grad(ro, ri, gm, dx.view(T, P), do)
    R, Y, GM, LG = (t.double().requires_grad_(True) for t in (r, y0, gm, lg))
    s = R + Y
    X = GM * s * (s.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    hh = X.view(T, H, d)
    cum = LG.cumsum(0)
    dec = (cum[:, None] - cum[None]).masked_fill(torch.ones(T, T, dtype=torch.bool, device="cuda").triu(1)[..., None],
                                                 -math.inf).exp()
    sc = (hh.transpose(0, 1).contiguous() @ hh.permute(1, 2, 0).contiguous()) * dec.permute(2, 0, 1) * 0.1
    att = (sc @ hh.transpose(0, 1).contiguous()).transpose(0, 1).reshape(T, P)
    ((s + att) * do.double()).sum().backward()
    for name, got, want in (("y", y.view(T, P), att.detach()), ("dr", dr, R.grad), ("dnorm_scale", ds, GM.grad),
                            ("dlog_decay", gr["dlog_decay"], LG.grad)):
        # fp32 throughout: sums of some hundred terms twice over
        err = float((got.double() - want).square().mean().sqrt() / want.square().mean().sqrt())
        say(f"  {name}: {err:.2e}")
        assert err <= 2.0 ** -18, name
    n = agm.clip_grads([{"dr": dr, "ds": ds}, {"dlog_decay": gr["dlog_decay"]}], 1.0)
    want = math.sqrt(sum(float(t.square().sum()) for t in (R.grad, GM.grad, LG.grad)))
    assert abs(float(n) - want) <= 2.0 ** -18 * want
    have = math.sqrt(sum(float(t.double().square().sum()) for t in (dr, ds, gr["dlog_decay"])))
    assert abs(have - 1.0) <= 2.0 ** -20
