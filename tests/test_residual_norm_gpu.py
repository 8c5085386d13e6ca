"""The residual step with its norms on the GPU, forward and backward, against the
definitions in 64 bits.

Tolerances.  As for layer norm: a float32 sum is off by at most DEPTH 2^-24 times
the sum of the magnitudes, DEPTH the longest chain of additions (a thread's columns,
at most 70, two trees of five levels, 32 warps; 256 covers every size here), so that
a normalised value is off by `off` below.  An error of n, y or dx goes on through
the formulas; each formula's own handful of roundings counts 8 2^-24 of its terms'
magnitudes.  A column sum over R rows has at most R + 256 additions in a chain.  On
top comes one rounding to the element type for each result."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import OlcError, ResidualNormPlan, residual_norm
from layers_ref import DTYPES, F32, ROUND, TINY, TORCH, Guarded, assert_near, normal

pytestmark = pytest.mark.gpu

DEPTH, EPS = 256, 1e-5
#: one element; odd widths; every number of warps and packs a row; rows of blocks' widths
#: and wider; more rows than blocks
SIZES = [(1, 1), (3, 2), (5, 31), (7, 128), (700, 96), (4, 1001), (33, 4096), (1300, 512), (2, 12000), (3, 20000), (2, 40000),
         (650, 2049), (640, 1024), (620, 4096), (310, 5120), (9, 4104)]
#: norm, after, gate, bias
FORMS = [("layer", True, "element", True), ("rms", True, "none", False), ("layer", False, "channel", True),
         ("rms", False, "none", False), ("rms", True, "channel", True)]


def inputs(rows, cols, dtype, form, seed=0):
    norm, after, gate, bias = form
    s = {"x": normal((rows, cols), dtype, seed + 1, 1.5, 0.25), "f": normal((rows, cols), dtype, seed + 2, 0.7, 0.1),
         "gamma": normal((cols,), dtype, seed + 3, 0.2, 1.0)}
    if bias:
        s["beta"] = normal((cols,), dtype, seed + 4, 0.2)
    if after:
        s["after_gamma"] = normal((cols,), dtype, seed + 5, 0.2, 1.0)
        if bias:
            s["after_beta"] = normal((cols,), dtype, seed + 6, 0.2)
    if gate != "none":
        s["gate"] = normal((cols,) if gate == "channel" else (rows, cols), dtype, seed + 7, 0.3, 0.5)
    return s


def stats_of(v, norm, eps=EPS):
    mean = v.mean(-1, keepdim=True) if norm == "layer" else torch.zeros_like(v[:, :1])
    return mean, 1 / torch.sqrt(((v - mean) ** 2).mean(-1, keepdim=True) + eps)


def off_of(v, hat, rstd):
    return DEPTH * F32 * (rstd * v.abs().mean(-1, keepdim=True) + hat.abs() + 1)


def forward_want(s, form, scale):
    """y, z, stats and the bounds of y's and z's errors before their rounding."""
    norm, after, gate, bias = form
    d = {k: v.double() for k, v in s.items()}
    f, stats, e_n = d["f"], [], torch.zeros_like(d["f"])
    n = f
    if after:
        mean, rstd = stats_of(f, norm)
        hat = (f - mean) * rstd
        n = hat * d["after_gamma"] + d.get("after_beta", 0)
        e_n = off_of(f, hat, rstd) * d["after_gamma"].abs() + 8 * F32 * ((hat * d["after_gamma"]).abs() + n.abs())
        stats = [mean[:, 0], rstd[:, 0]]
    g = d.get("gate", torch.ones(()))
    y = d["x"] + scale * g * n
    e_y = (scale * g).abs() * e_n + 8 * F32 * (d["x"].abs() + (scale * g * n).abs())
    mean, rstd = stats_of(y, norm)
    hat = (y - mean) * rstd
    z = hat * d["gamma"] + d.get("beta", 0)
    worst = e_y.max(-1, keepdim=True).values
    e_hat = rstd * (e_y + worst * (1 + hat.abs())) + off_of(y, hat, rstd)
    return y, z, [mean[:, 0], rstd[:, 0]] + stats, e_y, e_hat * d["gamma"].abs() + 8 * F32 * z.abs()


def vector(v, dtype, offset=0):
    return None if v is None else Guarded(1, v.numel(), dtype, None, offset, v.view(1, -1)).t.view(-1)


def run_forward(s, dtype, form, scale=0.5, pitch=None, offset=0, same=False):
    rows, cols = s["x"].shape
    norm, after, gate, bias = form
    m = lambda v=None: Guarded(rows, cols, dtype, pitch, offset, v)  # noqa: E731
    x, f = m(s["x"]), m(s["f"])
    y, z = (x, f) if same else (m(), m())
    gate_t = None if gate == "none" else (m(s["gate"]).t if gate == "element" else vector(s["gate"], dtype, offset))
    stats = Guarded(1, (4 if after else 2) * rows, "float32")
    with ResidualNormPlan(rows, cols, dtype, EPS, scale, norm, after) as plan:
        plan.forward(x.t, f.t, y.t, Z=z.t, gate=gate_t, stats=stats.t.view(-1),
                     **{k: vector(s.get(k), dtype, offset) for k in ("gamma", "beta", "after_gamma", "after_beta")})
        torch.cuda.synchronize()
    for g in (x, f, y, z, stats):
        g.check_guards()
    return y.t, z.t, stats.t.view(-1, rows)


def check_forward(s, dtype, form, scale=0.5, **kw):
    y, z, stats = run_forward(s, dtype, form, scale, **kw)
    want_y, want_z, want_stats, e_y, e_z = forward_want(s, form, scale)
    assert_near(y, want_y, e_y + ROUND[dtype] * (want_y.abs() + e_y) + TINY[dtype], "y")
    assert_near(z, want_z, e_z + ROUND[dtype] * (want_z.abs() + e_z) + TINY[dtype], "z")
    for i, w in enumerate(want_stats):
        v = want_y if i < 2 else s["f"].double()
        e = (e_y.max(-1).values if i < 2 else 0) + DEPTH * F32 * v.abs().mean(-1)
        rstd = want_stats[i | 1]
        assert_near(stats[i], w, e + 2.0 ** -149 if i % 2 == 0 else rstd * (rstd * e + DEPTH * F32), "stats %d" % i)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("form", FORMS)
def test_forward(rows, cols, form, dtype):
    check_forward(inputs(rows, cols, dtype, form), dtype, form)


#: rows of 16-bit elements on 4-byte boundaries
EVEN = [(40, 1002), (3, 5002), (700, 94), (2, 40002), (160, 2)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,cols", EVEN)
@pytest.mark.parametrize("form", FORMS)
def test_rows_of_pairs(rows, cols, form, dtype):
    check_forward(inputs(rows, cols, dtype, form), dtype, form)
    check_backward(rows, cols, dtype, form)
    check_forward(inputs(rows, cols, dtype, form), dtype, form, pitch=cols + 2, offset=2)
    check_backward(rows, cols, dtype, form, pitch=cols + 6, offset=6)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pitch,offset", [(1040, 0), (1033, 0), (1032, 1), (1032, 8)])
@pytest.mark.parametrize("same", [False, True])
def test_forward_pitches(pitch, offset, same, dtype):
    form = FORMS[0]
    check_forward(inputs(30, 1024, dtype, form), dtype, form, pitch=pitch, offset=offset, same=same)


@pytest.mark.parametrize("cols", [40000, 2048, 7])
def test_forward_in_place(cols):
    for form in FORMS[:2]:
        check_forward(inputs(5, cols, "bfloat16", form), "bfloat16", form, same=True)


@pytest.mark.parametrize("cols", [64, 1000, 4096, 40000])
def test_rows_far_from_zero(cols):
    """The mean of rows whose spread is small beside it keeps its digits: exact for
    equal values, whose normalised rows are the bias."""
    form = ("layer", True, "none", True)
    s = inputs(4, cols, "float32", form)
    s["f"] = torch.full((4, cols), 1234.56789)
    s["x"] = torch.full((4, cols), -777.7)
    s["after_beta"] = torch.full((cols,), 0.25)
    y, z, stats = run_forward(s, "float32", form, 1.0)
    assert (y == torch.full((4, cols), -777.7).cuda() + 0.25).all()
    assert torch.equal(z.cpu(), s["beta"].expand(4, cols))
    s["f"] = s["f"] + normal((4, cols), "float32", 3, 0.01)
    n = (run_forward(dict(s, x=torch.zeros(4, cols)), "float32", form, 1.0)[0]).double().cpu()
    d = s["f"].double()
    mean, rstd = stats_of(d, "layer")
    want = (d - mean) * rstd * s["after_gamma"].double() + 0.25
    # two roundings of the mean (2^-24 of it) times rstd, below 2^-24 1300 / 0.01
    assert float((n - want).abs().max()) < 4 * F32 * 1300 * float(rstd.max())


def test_infinities_and_nan_stay_in_their_rows():
    for norm in ("layer", "rms"):
        form = (norm, True, "none", False)
        s = inputs(6, 300, "float32", form)
        s["f"][1, 7], s["f"][3, 0], s["x"][4, 299] = float("inf"), float("nan"), float("-inf")
        y, z, _ = run_forward(s, "float32", form)
        clean = torch.tensor([True, False, True, False, False, True])
        assert torch.isfinite(z.cpu()[clean]).all() and torch.isnan(z.cpu()[~clean]).any(1).all()
        want = forward_want(s, form, 0.5)
        assert torch.equal(torch.isnan(y.cpu()), torch.isnan(want[0]))
        assert torch.equal(torch.isnan(z.cpu()), torch.isnan(want[1]))


def backward_want(s, form, scale, stats, dy, dz):
    """Gradients and bounds of their errors before the rounding, from the given stats."""
    norm, after, gate, bias = form
    d = {k: v.double() for k, v in s.items()}
    rows = d["f"].shape[0]
    stats = stats.double().cpu()
    zero = torch.zeros_like(d["f"])
    mean_of = lambda v: v.mean(-1, keepdim=True)  # noqa: E731

    def through(v, e_v, hat, rstd):
        m1 = mean_of(v) if norm == "layer" else 0 * mean_of(v)
        m2 = mean_of(v * hat)
        a1, a2 = mean_of(v.abs()), mean_of((v * hat).abs())
        size = rstd * (v.abs() + a1 + hat.abs() * a2)
        e = rstd * (e_v + mean_of(e_v) + hat.abs() * mean_of(e_v * hat.abs()))
        return rstd * (v - m1 - hat * m2), e + (8 + DEPTH) * F32 * size

    def column(v, e):
        return v.sum(0), e.sum(0) + (rows + 256) * F32 * v.abs().sum(0)

    out = {}
    dyd = zero if dy is None else dy.double()
    dx, e_dx = dyd, 2 * F32 * dyd.abs()
    if dz is not None:
        dzd = dz.double()
        mean, rstd = stats[0][:, None], stats[1][:, None]
        hat = (d["y"] - mean) * rstd
        g, e = through(dzd * d["gamma"], 2 * F32 * (dzd * d["gamma"]).abs(), hat, rstd)
        dx, e_dx = dx + g, e_dx + e + 4 * F32 * g.abs()
        out["dgamma"] = column(dzd * hat, 8 * F32 * (dzd * hat).abs())
        out["dbeta"] = column(dzd, zero)
    out["dx"] = dx, e_dx
    gs = scale * d.get("gate", torch.ones(()))
    dn, e_dn = gs * dx, gs.abs() * e_dx + 4 * F32 * (gs * dx).abs()
    n, e_n = d["f"], zero
    if after:
        mean, rstd = stats[2][:, None], stats[3][:, None]
        hat = (d["f"] - mean) * rstd
        ag = d["after_gamma"]
        n = hat * ag + d.get("after_beta", 0)
        e_n = 8 * F32 * ((hat * ag).abs() + n.abs())
        out["dafter_gamma"] = column(dn * hat, e_dn * hat.abs() + 8 * F32 * (dn * hat).abs())
        out["dafter_beta"] = column(dn, e_dn)
        out["df"] = through(dn * ag, e_dn * ag.abs() + 2 * F32 * (dn * ag).abs(), hat, rstd)
    else:
        out["df"] = dn, e_dn
    if gate != "none":
        v = scale * n * dx
        e = abs(scale) * (n.abs() * e_dx + e_n * dx.abs()) + 8 * F32 * v.abs()
        out["dgate"] = column(v, e) if gate == "channel" else (v, e)
    return out


def make_backward(rows, cols, dtype, form, seed=0):
    s = inputs(rows, cols, dtype, form, seed)
    s["y"] = normal((rows, cols), dtype, seed + 8, 1.7, 0.25)
    stats = [v[:, 0] for v in stats_of(s["y"].double(), form[0])]
    if form[1]:
        stats += [v[:, 0] for v in stats_of(s["f"].double(), form[0])]
    return s, torch.stack(stats).float(), normal((rows, cols), dtype, seed + 9), normal((rows, cols), dtype, seed + 10)


def run_backward(s, stats, dy, dz, dtype, form, scale=0.5, pitch=None, offset=0, same=False, skip=(), plan=None):
    rows, cols = s["f"].shape
    norm, after, gate, bias = form
    m = lambda v=None: Guarded(rows, cols, dtype, pitch, offset, v)  # noqa: E731
    mats = {k: None if v is None else m(v) for k, v in (("dy", dy), ("dz", dz), ("f", s["f"]), ("y", s["y"]))}
    names = ["dx", "df"] + (["dgamma", "dbeta"] if dz is not None else []) + (
        ["dafter_gamma", "dafter_beta"] if after else []) + (["dgate"] if gate != "none" else [])
    out = {}
    for k in names:
        if k in skip:
            continue
        matrix = k in ("dx", "df") or (k == "dgate" and gate == "element")
        out[k] = m() if matrix else Guarded(1, cols, dtype, None, offset)
    gate_m = m(s["gate"]) if gate == "element" else None
    if same:
        out["dx"], out["df"] = mats["dy"], mats["f"]
        if gate_m:
            out["dgate"] = gate_m
    t = lambda g: None if g is None else g.t  # noqa: E731
    arg = {k: (g.t if g.t.shape == (rows, cols) and (k in ("dx", "df") or (k == "dgate" and gate == "element"))
               else g.t.view(-1)) for k, g in out.items()}
    own = plan or ResidualNormPlan(rows, cols, dtype, EPS, scale, norm, after)
    own.backward(t(mats["dy"]), t(mats["dz"]), mats["f"].t, mats["y"].t, stats.cuda(),
                 gate=t(gate_m) if gate == "element" else vector(s.get("gate"), dtype, offset),
                 dX=arg.get("dx"), dF=arg.get("df"),
                 **{k: vector(s.get(k), dtype, offset) for k in ("gamma", "after_gamma", "after_beta")},
                 **{k: arg.get(k) for k in ("dgate", "dgamma", "dbeta", "dafter_gamma", "dafter_beta")})
    torch.cuda.synchronize()
    if plan is None:
        own.close()
    for g in list(mats.values()) + list(out.values()) + [gate_m]:
        if g is not None:
            g.check_guards()
    return {k: v.clone() for k, v in arg.items()}


def check_backward(rows, cols, dtype, form, scale=0.5, dy=True, dz=True, **kw):
    s, stats, dyv, dzv = make_backward(rows, cols, dtype, form)
    dyv, dzv = dyv if dy else None, dzv if dz else None
    got = run_backward(s, stats, dyv, dzv, dtype, form, scale, **kw)
    want = backward_want(s, form, scale, stats, dyv, dzv)
    for k, v in got.items():
        w, e = want[k]
        assert_near(v, w, e + ROUND[dtype] * (w.abs() + e) + TINY[dtype], k)
    return got


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("form", FORMS)
def test_backward(rows, cols, form, dtype):
    check_backward(rows, cols, dtype, form)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1024, 5120])
@pytest.mark.parametrize("extra,offset", [(16, 0), (9, 0), (8, 1), (8, 8)])
@pytest.mark.parametrize("same", [False, True])
def test_backward_pitches(extra, offset, same, cols, dtype):
    check_backward(30, cols, dtype, FORMS[0], pitch=cols + extra, offset=offset, same=same)


@pytest.mark.parametrize("cols", [96, 1001, 4096, 5120])
@pytest.mark.parametrize("form", FORMS)
def test_backward_without_one_of_the_gradients(cols, form):
    check_backward(40, cols, "bfloat16", form, dy=False)
    check_backward(40, cols, "bfloat16", form, dz=False)


@pytest.mark.parametrize("cols", [96, 4096, 5120])
@pytest.mark.parametrize("form", FORMS[:3])
def test_backward_of_some_outputs(cols, form):
    names = ["dx", "df", "dgamma", "dbeta", "dafter_gamma", "dafter_beta", "dgate"]
    s, stats, dy, dz = make_backward(200, cols, "float32", form)
    norm, after, gate, bias = form
    with ResidualNormPlan(200, cols, "float32", EPS, 0.5, norm, after) as plan:
        every = run_backward(s, stats, dy, dz, "float32", form, plan=plan)
        want = backward_want(s, form, 0.5, stats, dy, dz)
        for k in every:
            only = run_backward(s, stats, dy, dz, "float32", form, skip=[n for n in names if n != k], plan=plan)
            assert list(only) == [k]
            w, e = want[k]
            assert_near(only[k], w, e + ROUND["float32"] * (w.abs() + e) + TINY["float32"], k)
        again = run_backward(s, stats, dy, dz, "float32", form, plan=plan)
        assert all(torch.equal(again[k], every[k]) for k in every)


def test_gradients_against_differences():
    form = ("layer", True, "element", True)
    rows, cols, scale = 3, 9, 0.7
    s = inputs(rows, cols, "float32", form)
    cy, cz = normal((rows, cols), "float32", 21), normal((rows, cols), "float32", 22)
    keys = {"x": "dx", "f": "df", "gate": "dgate", "gamma": "dgamma", "beta": "dbeta", "after_gamma": "dafter_gamma",
            "after_beta": "dafter_beta"}

    def value(v):
        y, z, _ = run_forward(v, "float32", form, scale)
        return float((y.double().cpu() * cy.double()).sum() + (z.double().cpu() * cz.double()).sum())

    y, z, stats = run_forward(s, "float32", form, scale)
    got = run_backward(dict(s, y=y.cpu()), stats.cpu(), cy, cz, "float32", form, scale)
    for k, dk in keys.items():
        for at in [0, s[k].numel() // 2, s[k].numel() - 1]:
            h = 2.0 ** -6
            up, down = {q: v.clone() for q, v in s.items()}, {q: v.clone() for q, v in s.items()}
            up[k].view(-1)[at] += h
            down[k].view(-1)[at] -= h
            slope = (value(up) - value(down)) / (2 * h)
            # h^2 of the third derivatives, and roundings of the values over h
            assert abs(slope - float(got[dk].reshape(-1)[at])) < 2e-2 * (1 + abs(slope)), (k, at)


def test_rows_of_nothing():
    with ResidualNormPlan(0, 8, "float32", after=True) as plan:
        e = torch.empty(0, 8, device="cuda")
        plan.forward(e, e, e, Z=e)
        ones = [torch.ones(8, device="cuda") for _ in range(5)]
        plan.backward(e, e, e, e, torch.empty(0, device="cuda"), gate=torch.ones(8, device="cuda"), dX=e, dF=e,
                      dgate=ones[0], dgamma=ones[1], dbeta=ones[2], dafter_gamma=ones[3], dafter_beta=ones[4])
        assert all(float(o.abs().sum()) == 0 for o in ones)


def test_without_a_norm_behind():
    s = inputs(50, 640, "bfloat16", FORMS[1])
    with ResidualNormPlan(50, 640, "bfloat16", EPS, 1.0, "rms", True) as plan:
        y, z = torch.empty(50, 640, dtype=torch.bfloat16, device="cuda"), torch.empty(50, 640, dtype=torch.bfloat16, device="cuda")
        only = torch.empty_like(y)
        plan.forward(s["x"].cuda(), s["f"].cuda(), y, Z=z, after_gamma=s["after_gamma"].cuda())
        plan.forward(s["x"].cuda(), s["f"].cuda(), only, after_gamma=s["after_gamma"].cuda())
        assert torch.equal(y, only)


def test_one_shot_graph_and_streams():
    form = FORMS[0]
    s, stats, dy, dz = make_backward(64, 512, "float16", form)
    c = {k: v.cuda() for k, v in s.items()}
    y, z = residual_norm(c["x"].view(4, 16, 512), c["f"].view(4, 16, 512), c["gamma"], c["beta"], c["gate"].view(4, 16, 512),
                         c["after_gamma"], c["after_beta"], scale=0.5, after=True)
    want = run_forward(s, "float16", form)
    assert torch.equal(y.view(64, 512), want[0]) and torch.equal(z.view(64, 512), want[1])
    with ResidualNormPlan(64, 512, "float16", EPS, 0.5, "layer", True) as plan:
        dx, df = torch.empty_like(c["x"]), torch.empty_like(c["x"])
        dg = torch.empty_like(c["gamma"])
        args = (dy.cuda(), dz.cuda(), c["f"], c["y"], stats.cuda())
        call = lambda: plan.backward(*args, gate=c["gate"], gamma=c["gamma"], after_gamma=c["after_gamma"], dX=dx, dF=df, dgamma=dg)  # noqa: E731
        call()
        first = [t.clone() for t in (dx, df, dg)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        for t in (dx, df, dg):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((dx, df, dg), first))


def test_offsets_beyond_32_bits():
    rows, cols = 530_000, 4096
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    last = normal((2, cols), "bfloat16", 1).cuda()
    x[-2:] = last
    with ResidualNormPlan(rows, cols, "bfloat16", EPS, 1.0, "rms") as plan, ResidualNormPlan(2, cols, "bfloat16", EPS, 1.0, "rms") as two:
        stats, s2 = torch.empty(2, rows, device="cuda"), torch.empty(2, 2, device="cuda")
        y, z, y2, z2 = torch.empty_like(x), torch.empty_like(x), torch.empty_like(last), torch.empty_like(last)
        plan.forward(x, x, y, Z=z, stats=stats)
        two.forward(last, last, y2, Z=z2, stats=s2)
        assert torch.equal(y[-2:], y2)
        # other launch shapes for two rows: other orders of the sums, two roundings at most
        assert float((z[-2:].double() - z2.double()).abs().max()) <= 2 * 2.0 ** -8 * float(z2.abs().max())
        dx, dx2 = torch.empty_like(x), torch.empty_like(last)
        plan.backward(None, z, None, y, stats, dX=dx)
        two.backward(None, z[-2:].contiguous(), None, y2, stats[:, -2:].contiguous(), dX=dx2)
        assert float((dx[-2:].double() - dx2.double()).abs().max()) <= 2 * 2.0 ** -8 * float(dx2.abs().max())


def test_refusals():
    with ResidualNormPlan(4, 8, "float16", after=True) as plan:
        t = lambda *s, of=torch.float16: torch.zeros(s, dtype=of, device="cuda")  # noqa: E731
        x, f, y, stats = t(4, 8), t(4, 8), t(4, 8), t(4, 4, of=torch.float32)
        for kw in [{"gate": t(4, 7)}, {"gate": t(7)}, {"gamma": t(7)}, {"Z": t(4, 9)}, {"stats": t(2, 4, of=torch.float32)}]:
            with pytest.raises(ValueError):
                plan.forward(x, f, y, **kw)
        with pytest.raises(TypeError):
            plan.forward(x, f.float(), y)
        with pytest.raises(ValueError):
            plan.backward(x, None, f, None, stats, gate=t(8), dgate=t(4, 8))
        for args, kw in [((None, None, f, y, stats), {"dX": x}), ((x, None, f, y, stats), {"dgamma": t(8)}),
                         ((x, None, f, y, stats), {"dgate": t(8)}), ((x, None, None, y, stats), {"dX": x}),
                         ((x, y, f, None, stats), {"dX": x}), ((x, y, f, y, None), {"dX": x})]:
            with pytest.raises(OlcError) as e:
                plan.backward(*args, **kw)
            assert e.value.name == "OLC_ERR_NULL"
    with ResidualNormPlan(4, 8, "float16") as plan:
        with pytest.raises(OlcError) as e:
            plan.backward(x, None, f, None, None, dafter_gamma=t(8))
        assert e.value.name == "OLC_ERR_INVALID"
        lib, h, p = plan.lib, plan._h, x.data_ptr()
        call = lambda *a: lib.olc_residual_norm_forward(h, *a)  # noqa: E731
        rest = (None, None, None, None)
        assert call(p, 7, p, 8, None, 0, *rest, p, 8, None, 8, None, None) == 13
        assert call(p, 8, p, 8, p, 7, *rest, p, 8, None, 8, None, None) == 13
        assert call(p + 1, 8, p, 8, None, 0, *rest, p, 8, None, 8, None, None) == 13
        assert call(p, 8, None, 8, None, 0, *rest, p, 8, None, 8, None, None) == 1
