"""GELU's tail in the gated product: where the distribution function is small
it is still good to 2^-16 of itself (the products multiply it by any u), on
every kernel that forms it.

Tolerances: one rounding to the type (gradient: two), 2^-16 of the value for
the activation, and nothing absolute.  The products have one term, so g and u
are exact."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import GatedPlan
from layers_ref import ROUND, TINY, TORCH, assert_near

pytestmark = pytest.mark.gpu

F64 = torch.float64
ROOT_HALF = 0.5 ** 0.5


def gelu(g):
    return 0.5 * g * torch.special.erfc(-g * ROOT_HALF)


def gates(dtype, count, low):
    return torch.linspace(low, -0.5, count).to(TORCH[dtype])


@pytest.mark.parametrize("dtype,low,big", [("bfloat16", -12.5, 2.0 ** 60), ("float16", -5.5, 60000.0), ("float32", -12.5, 2.0 ** 60)])
# rows of the few-row kernel, of single CTAs and pairs, and a K of zeros that is cut into slices
@pytest.mark.parametrize("m,d", [(1, 8), (40, 8), (300, 8), (3000, 8), (130, 4096)])
@pytest.mark.parametrize("trans_w", [False, True])
def test_gelu_tail_forward(m, d, trans_w, dtype, low, big):
    f = 520
    t = TORCH[dtype]
    x = torch.zeros(m, d, dtype=t)
    x[:, 0] = 1
    wg, wu = torch.zeros(d, f, dtype=t), torch.zeros(d, f, dtype=t)
    wg[0], wu[0] = gates(dtype, f, low), big
    h = torch.empty(m, f, dtype=t, device="cuda")
    w = [(v.t().contiguous() if trans_w else v).cuda() for v in (wg, wu)]
    with GatedPlan(m, d, f, dtype, "gelu", trans_w) as plan:
        plan.forward(x.cuda(), *w, h)
        torch.cuda.synchronize()
    want = (gelu(wg[0].to(F64)) * float(wu[0, 0])).expand(m, f)
    # (what underflows to the type's subnormals: half of the smallest one)
    assert_near(h, want, (ROUND[dtype] + 2.0 ** -16) * want.abs() + TINY[dtype], "h")


@pytest.mark.parametrize("dtype,low,big", [("bfloat16", -12.5, 2.0 ** 60), ("float16", -5.5, 60000.0), ("float32", -12.5, 2.0 ** 60)])
@pytest.mark.parametrize("cols", [1, 2, 8])
def test_gelu_tail_backward(cols, dtype, low, big):
    # one hidden unit of `cols`; Wg = 0, so dX = du Wu = dh act(g) in every row; with Wu = 0, dX = dg Wg
    m, t = 600, TORCH[dtype]
    g = torch.zeros(m, cols, dtype=t)
    g[:, 0] = gates(dtype, m, low)
    dh = torch.zeros(m, cols, dtype=t)
    dh[:, 0] = big
    u = torch.ones(m, cols, dtype=t)
    one, zero = torch.zeros(1, cols, dtype=t), torch.zeros(1, cols, dtype=t)
    one[0, 0] = 1
    x, dx = torch.ones(m, 1, dtype=t).cuda(), torch.empty(m, 1, dtype=t, device="cuda")
    gd = g[:, 0].to(F64)
    slope = 0.5 * torch.special.erfc(-gd * ROOT_HALF) + gd * torch.exp(-0.5 * gd * gd) * 0.3989422804014327
    terms = 0.5 * torch.special.erfc(-gd * ROOT_HALF).abs() + gd.abs() * torch.exp(-0.5 * gd * gd) * 0.3989422804014327
    with GatedPlan(m, 1, cols, dtype, "gelu") as plan:
        plan.backward(dh.cuda(), x, zero.cuda(), one.cuda(), g.cuda(), u.cuda(), dX=dx)
        want = gelu(gd) * float(dh[0, 0])
        assert_near(dx[:, 0], want, (2 * ROUND[dtype] + 2.0 ** -15) * want.abs() + 2 * TINY[dtype], "du")
        plan.backward(dh.cuda(), x, one.cuda(), zero.cuda(), g.cuda(), u.cuda(), dX=dx)
        want = slope * float(dh[0, 0])
        # (its two terms cancel at g = -0.75: each is good to 2^-16 of itself)
        assert_near(dx[:, 0], want, 2 * ROUND[dtype] * want.abs() + 2.0 ** -15 * terms * float(dh[0, 0]) + 2 * TINY[dtype], "dg")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
def test_gelu_ends_and_middle(dtype):
    # zero, infinity, NaN, beyond what the exponential reaches, and the positive side
    t = TORCH[dtype]
    v = torch.tensor([0.0, -0.0, 0.5, 1.0, 3.0, 9.0, 100.0, 60000.0, -14.0, -30.0, -300.0, -60000.0], dtype=t)
    x = torch.ones(3, 1, dtype=t)
    x[2] = float("nan")
    h = torch.empty(3, v.numel(), dtype=t, device="cuda")
    with GatedPlan(3, 1, v.numel(), dtype, "gelu") as plan:
        plan.forward(x.cuda(), v.view(1, -1).cuda(), torch.ones(1, v.numel(), dtype=t).cuda(), h)
    want = gelu(v.to(F64)).expand(2, -1)
    assert_near(h[:2], want, (ROUND[dtype] + 2.0 ** -16) * want.abs() + 1e-37 + TINY[dtype], "h")
    assert torch.isnan(h[2]).all()
