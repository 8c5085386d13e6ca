"""Layer norm on the GPU, forward and backward, against the definition in 64
bits.

Tolerances.  A float32 sum of terms t_j, in whatever order a block takes, is
off by at most DEPTH * 2^-24 * sum |t_j|, with DEPTH the longest chain of
additions: a thread's own elements (at most 16 packs of 8, or a 1024th of a
long row) plus two trees of five levels; 256 covers every size here.  The
error of the mean therefore moves xh = (x - mean) rstd by at most
DEPTH 2^-24 rstd mean|x|, that of the variance by DEPTH 2^-24 |xh| (half of
2 DEPTH, the square root halving it), and a handful of roundings more are
within the same factor.  On top comes the one rounding to the element type."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import LayerNormPlan, OlcError, layer_norm
from layers_ref import DTYPES, F32, ROUND, TINY, TORCH, Guarded, assert_near, normal

pytestmark = pytest.mark.gpu

DEPTH = 256
EPS = 1e-5
SIZES = [(1, 1), (3, 2), (5, 31), (7, 128), (700, 96), (4, 1001), (33, 4096), (1300, 512), (2, 12000), (9, 16384),
         (3, 20000), (2, 70001), (650, 2049)]
# shapes of the kernels for many rows: short rows, rings of rows of full and of other widths, wide rows
MANY = [(5000, 128), (4900, 40), (4870, 256), (700, 1024), (640, 1040), (610, 4096), (320, 12000), (310, 16384)]


def reference(x, gamma, beta, eps=EPS):
    """y, mean, rstd and the scale of xh's error, in float64 from the given inputs."""
    x = x.double()
    n = x.shape[-1]
    mean = x.sum(-1, keepdim=True) / n
    rstd = 1 / torch.sqrt(((x - mean) ** 2).sum(-1, keepdim=True) / n + eps)
    xh = (x - mean) * rstd
    g = 1.0 if gamma is None else gamma.double()
    b = 0.0 if beta is None else beta.double()
    off = DEPTH * F32 * (rstd * x.abs().mean(-1, keepdim=True) + xh.abs() + 1)
    return xh * g + b, mean[:, 0], rstd[:, 0], xh, off


def run_forward(x, gamma, beta, dtype, pitch=None, offset=0, stats=True, eps=EPS, same=False):
    rows, cols = x.shape
    gx = Guarded(rows, cols, dtype, pitch, offset, x)
    gy = gx if same else Guarded(rows, cols, dtype, pitch, offset)
    gm, gr = (Guarded(1, rows, "float32") for _ in range(2))
    gg, gb = (None if v is None else Guarded(1, cols, dtype, None, offset, v.view(1, -1)).t.view(-1)
              for v in (gamma, beta))
    with LayerNormPlan(rows, cols, dtype, eps) as plan:
        plan.forward(gx.t, gg, gb, gy.t, mean=gm.t.view(-1) if stats else None, rstd=gr.t.view(-1) if stats else None)
        torch.cuda.synchronize()
    for g in (gx, gy, gm, gr):
        g.check_guards()
    return gy.t, gm.t[0], gr.t[0]


def check_forward(x, gamma, beta, dtype, eps=EPS, **kw):
    y, mean, rstd = run_forward(x, gamma, beta, dtype, eps=eps, **kw)
    want, m, r, xh, off = reference(x, gamma, beta, eps)
    g = 1.0 if gamma is None else gamma.double().abs()
    b = 0.0 if beta is None else beta.double().abs()
    assert_near(y, want, ROUND[dtype] * want.abs() + (1 + ROUND[dtype]) * (off * g + 4 * F32 * b) + TINY[dtype], "y")
    assert_near(mean, m, DEPTH * F32 * x.double().abs().mean(-1) + TINY["float32"], "mean")
    # rstd' = -rstd^3 / 2 var': the variance is off by DEPTH 2^-24 of itself, and by the mean's error squared
    dm = DEPTH * F32 * x.double().abs().mean(-1)
    assert_near(rstd, r, r * (DEPTH * F32 + (r * dm) ** 2), "rstd")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES + MANY)
def test_forward(rows, cols, dtype):
    x = normal((rows, cols), dtype, 1, 1.5, 0.25)
    gamma, beta = normal((cols,), dtype, 2, 0.3, 1.0), normal((cols,), dtype, 3, 0.3)
    check_forward(x, gamma, beta, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,pitch,offset", [(256, 264, 0), (256, 257, 0), (256, 256, 1), (1024, 1024, 3), (100, 128, 8)])
def test_forward_pitches_and_offsets(cols, pitch, offset, dtype):
    x = normal((37, cols), dtype, 4)
    gamma, beta = normal((cols,), dtype, 5, 0.3, 1.0), normal((cols,), dtype, 6)
    check_forward(x, gamma, beta, dtype, pitch=pitch, offset=offset)
    check_forward(x, gamma, beta, dtype, pitch=pitch, offset=offset, same=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_forward_without_weights_or_statistics(dtype):
    x = normal((19, 333), dtype, 7)
    want, *_, off = reference(x, None, None)
    y, mean, rstd = run_forward(x, None, None, dtype, stats=False)
    assert_near(y, want, ROUND[dtype] * want.abs() + 2 * off, "y")
    assert (mean == 7.25).all() and (rstd == 7.25).all()
    check_forward(x, normal((333,), dtype, 8, 0.3, 1.0), None, dtype)
    check_forward(x, None, normal((333,), dtype, 9), dtype)


def test_rows_far_from_zero_keep_their_variance():
    # sum of squares minus squared sum would lose every digit here: 1000^2 2^-24 is above the variance's last digits
    check_forward(normal((8, 4096), "float32", 10, 1.0, 1000.0), None, None, "float32")
    check_forward(normal((8, 16400), "float32", 11, 1.0, -1000.0), None, None, "float32")


@pytest.mark.parametrize("cols", [64, 4096, 40000])
def test_equal_values_and_special_values_stay_in_their_rows(cols):
    x = normal((6, cols), "float32", 12)
    x[1] = 2.5
    x[2, cols // 2] = float("nan")
    x[3, 0] = float("inf")
    x[4] = 0.0
    beta = normal((cols,), "float32", 13)
    y, mean, rstd = (v.cpu() for v in run_forward(x, None, beta, "float32"))
    assert torch.equal(y[1], beta) and torch.equal(y[4], beta) and float(mean[1]) == 2.5
    assert torch.isnan(y[2]).all() and torch.isnan(y[3]).all() and float(mean[3]) == float("inf")
    want, *_, off = reference(x[[0, 5]], None, beta)
    assert_near(y[[0, 5]], want, F32 * want.abs() + off + 4 * F32 * beta.abs(), "the other rows")
    y, _, rstd = run_forward(x, None, None, "float32", eps=0.0)
    assert torch.isinf(rstd[1]) and torch.isnan(y[1]).all()


# ---- backward ------------------------------------------------------------------


def reference_grads(dy, x, gamma, mean, rstd):
    """dx, dgamma, dbeta and the scales of their errors, in float64 from the float32 statistics."""
    dy, x, mean, rstd = dy.double(), x.double(), mean.double()[:, None], rstd.double()[:, None]
    g = 1.0 if gamma is None else gamma.double()
    xh, dxh = (x - mean) * rstd, dy * g
    c1, c2 = dxh.mean(-1, keepdim=True), (dxh * xh).mean(-1, keepdim=True)
    dx = rstd * (dxh - c1 - xh * c2)
    # xh itself is off by 2 roundings of |x| rstd and of itself
    near = 4 * F32 * (rstd * (x.abs() + mean.abs()) + xh.abs())
    s1 = dxh.abs().mean(-1, keepdim=True)
    s2 = (dxh * xh).abs().mean(-1, keepdim=True)
    sx = rstd * (DEPTH * F32 * (dxh.abs() + s1 + xh.abs() * s2) + near * s2 + xh.abs() * (dxh.abs() * near).mean(-1, keepdim=True))
    # the longest chain of a column sum: a block's rows, then the blocks and shares
    depth = min(len(x), 64 + len(x) // 64) + 96
    sg = depth * F32 * (dy * xh).abs().sum(0) + (dy.abs() * near).sum(0)
    return dx, (dy * xh).sum(0), dy.sum(0), sx, sg, depth * F32 * dy.abs().sum(0)


def check_backward(rows, cols, dtype, pitch=None, offset=0, gamma=True, same=None):
    x, dy = normal((rows, cols), dtype, 21, 1.5, 0.25), normal((rows, cols), dtype, 22)
    gm = normal((cols,), dtype, 23, 0.3, 1.0) if gamma else None
    _, mean, rstd, _, _ = reference(x, None, None)
    mean, rstd = mean.float(), rstd.float()
    gx, gdy = Guarded(rows, cols, dtype, pitch, offset, x), Guarded(rows, cols, dtype, pitch, offset, dy)
    gdx = {"dy": gdy, "x": gx}.get(same) or Guarded(rows, cols, dtype, pitch, offset)
    dg, db = (Guarded(1, cols, dtype, None, offset) for _ in range(2))
    gg = None if gm is None else Guarded(1, cols, dtype, None, offset, gm.view(1, -1)).t.view(-1)
    with LayerNormPlan(rows, cols, dtype) as plan:
        plan.backward(gdy.t, gx.t, gg, mean.cuda(), rstd.cuda(), gdx.t, dgamma=dg.t.view(-1), dbeta=db.t.view(-1))
        torch.cuda.synchronize()
    for g in (gx, gdy, gdx, dg, db):
        g.check_guards()
    dx, wg, wb, sx, sg, sb = reference_grads(dy, x, gm, mean, rstd)
    u = ROUND[dtype]
    assert_near(gdx.t, dx, u * dx.abs() + (1 + u) * sx + TINY[dtype], "dx")
    assert_near(dg.t[0], wg, u * wg.abs() + (1 + u) * sg + TINY[dtype], "dgamma")
    assert_near(db.t[0], wb, u * wb.abs() + (1 + u) * sb + TINY[dtype], "dbeta")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SIZES + MANY + [(2600, 256), (1, 5000), (3000, 33)])
def test_backward(rows, cols, dtype):
    check_backward(rows, cols, dtype)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols,pitch,offset", [(256, 264, 0), (256, 257, 0), (256, 256, 1), (100, 128, 8), (17000, 17001, 1)])
def test_backward_pitches_and_offsets(cols, pitch, offset, dtype):
    check_backward(300, cols, dtype, pitch=pitch, offset=offset)
    check_backward(21, cols, dtype, pitch=pitch, offset=offset, gamma=False, same="dy")
    check_backward(21, cols, dtype, pitch=pitch, offset=offset, same="x")


@pytest.mark.parametrize("rows,cols", [(40, 96), (40, 18000), (0, 96), (620, 1040), (320, 10000)])
def test_backward_in_parts_and_with_no_rows(rows, cols):
    x, dy = normal((rows, cols), "float32", 24).cuda(), normal((rows, cols), "float32", 25).cuda()
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    whole = [torch.full_like(x, 9), torch.full((cols,), 9.0, device="cuda"), torch.full((cols,), 9.0, device="cuda")]
    with LayerNormPlan(rows, cols, "float32") as plan:
        plan.backward(dy, x, None, mean, rstd, *whole)
        for part in range(3):
            got = [torch.full_like(t, 9) if i == part else None for i, t in enumerate(whole)]
            plan.backward(dy, x, None, mean, rstd, *got)
            assert torch.equal(got[part], whole[part]), part
        plan.backward(dy, x, None, mean, rstd)
        if rows == 0:
            plan.forward(x, None, None, x, mean=mean, rstd=rstd)
            assert not whole[1].any() and not whole[2].any()


@pytest.mark.parametrize("rows,cols", [(640, 1040), (320, 9000)])
def test_backward_rings_in_place_and_without_gamma(rows, cols):
    check_backward(rows, cols, "bfloat16", gamma=False, same="dy")
    check_backward(rows, cols, "float32", pitch=cols + 8, same="x")


def test_backward_repeats_bit_for_bit_on_several_streams():
    rows, cols = 5000, 1024
    x, dy = normal((rows, cols), "bfloat16", 26).cuda(), normal((rows, cols), "bfloat16", 27).cuda()
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    with LayerNormPlan(rows, cols, "bfloat16") as plan:
        torch.cuda.synchronize()
        for i in range(9):      # every call writes the plan's partial sums: the plan orders the streams
            o = [torch.empty_like(x), torch.empty_like(x[0]), torch.empty_like(x[0])]
            torch.cuda.synchronize() if i < 2 else None
            plan.backward(dy if i % 2 else x, x, None, mean, rstd, *o, stream=streams[i % 3])
            outs.append(o)
        torch.cuda.synchronize()
    for i in range(2, 9):
        assert all(torch.equal(a, b) for a, b in zip(outs[i], outs[i % 2])), i


def test_gradients_match_central_differences():
    # L = sum w y in float64 from float32 outputs; along a direction v of norm sqrt(n) the central difference is
    # off by h^2 / 6 of the third derivative (a few times |w| for unit-variance rows) and by the outputs'
    # roundings over h; h = 2^-7 makes both below 2e-3 of |w| |v|
    rows, cols, h = 3, 40, 2.0 ** -7
    x, w = normal((rows, cols), "float32", 31).cuda(), normal((rows, cols), "float32", 32).cuda()
    gamma, beta = normal((cols,), "float32", 33, 0.3, 1.0).cuda(), normal((cols,), "float32", 34).cuda()
    with LayerNormPlan(rows, cols, "float32") as plan:
        def loss(a, g, b):
            y = torch.empty_like(a)
            plan.forward(a, g, b, y)
            return float((y.double() * w.double()).sum())

        mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        plan.forward(x, gamma, beta, torch.empty_like(x), mean=mean, rstd=rstd)
        dx, dg, db = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(beta)
        plan.backward(w, x, gamma, mean, rstd, dx, dg, db)
        for i, (at, grad) in enumerate(((x, dx), (gamma, dg), (beta, db))):
            for seed in range(4):
                v = normal(tuple(at.shape), "float32", 40 + seed).cuda()
                args = [x, gamma, beta]
                args[i] = at + h * v
                up = loss(*args)
                args[i] = at - h * v
                down = loss(*args)
                want = float((grad.double() * v.double()).sum())
                scale = float(w.double().norm() * v.double().norm())
                assert abs((up - down) / (2 * h) - want) <= 2e-3 * scale, (i, seed)


def test_offsets_beyond_32_bits():
    rows, cols, pitch = 3, 64, 2 ** 30 + 64
    storage = torch.empty(2 * pitch + cols, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(storage, (rows, cols), (pitch, 1))
    x.copy_(normal((rows, cols), "bfloat16", 51))
    y = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    dx = torch.empty_like(y)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    with LayerNormPlan(rows, cols, "bfloat16") as plan:
        plan.forward(x, None, None, y, mean=mean, rstd=rstd)
        plan.backward(x, x, None, mean, rstd, dx)
        dense = x.contiguous()
        y2, dx2 = torch.empty_like(y), torch.empty_like(y)
        plan.forward(dense, None, None, y2)
        plan.backward(dense, dense, None, mean, rstd, dx2)
        assert torch.equal(y, y2) and torch.equal(dx, dx2)


def test_captured_in_a_graph_and_one_shot():
    x = normal((64, 512), "float16", 61).cuda()
    dy = normal((64, 512), "float16", 62).cuda()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dg, db = torch.empty_like(x[0]), torch.empty_like(x[0])
    mean, rstd = torch.empty(64, device="cuda"), torch.empty(64, device="cuda")
    with LayerNormPlan(64, 512, "float16") as plan:
        def step():
            plan.forward(x, None, None, y, mean=mean, rstd=rstd)
            plan.backward(dy, x, None, mean, rstd, dx, dg, db)
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, dx, dg, db)]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for t in (y, dx, dg, db):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, (y, dx, dg, db)))
    assert torch.equal(layer_norm(x.view(8, 8, 512)).view(64, 512), want[0])


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    with LayerNormPlan(4, 8, "float32") as plan:
        for bad in (x.half(), x[:, :4], torch.zeros(4, 8), torch.zeros(8, 4, device="cuda").t()):
            with pytest.raises((TypeError, ValueError)):
                plan.forward(bad, None, None, x)
        with pytest.raises(ValueError):
            plan.forward(x, torch.zeros(7, device="cuda"), None, x)
        with pytest.raises(OlcError) as e:
            plan.backward(x, x, None, None, None, x)
        assert e.value.name == "OLC_ERR_NULL"
        lib, p = plan.lib, x.data_ptr()
        assert lib.olc_layer_norm_forward(plan._h, p, 7, None, None, p, 8, None, None, None) == 13
        assert lib.olc_layer_norm_forward(plan._h, p + 2, 8, None, None, p, 8, None, None, None) == 13
        assert lib.olc_layer_norm_forward(plan._h, None, 8, None, None, p, 8, None, None, None) == 1
        assert lib.olc_layer_norm_forward(None, p, 8, None, None, p, 8, None, None, None) == 1
