"""The sigmoid gate's slope s (1 - s) where s is close to 1: as small as e^-g,
and good to that.  Tolerances: two roundings to the type (dg's, dX's) and 2^-16
of the value for the activation."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import GatedPlan
from layers_ref import DTYPES, ROUND, TINY, TORCH, assert_near

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("cols", [1, 8])
def test_sigmoid_slope_on_both_sides(cols, dtype):
    # Wu = 0 and Wg = 1 at one hidden unit: dX = dg = dh u act'(g) in every row
    m, t = 600, TORCH[dtype]
    reach, big = (16.0, 60000.0) if dtype == "float16" else (80.0, 2.0 ** 40)
    g = torch.zeros(m, cols, dtype=t)
    g[:, 0] = torch.linspace(-reach, reach, m).to(t)
    dh = torch.zeros(m, cols, dtype=t)
    dh[:, 0] = big
    u = torch.ones(m, cols, dtype=t)
    one, zero = torch.zeros(1, cols, dtype=t), torch.zeros(1, cols, dtype=t)
    one[0, 0] = 1
    x, dx = torch.ones(m, 1, dtype=t).cuda(), torch.empty(m, 1, dtype=t, device="cuda")
    with GatedPlan(m, 1, cols, dtype, "sigmoid") as plan:
        plan.backward(dh.cuda(), x, one.cuda(), zero.cuda(), g.cuda(), u.cuda(), dX=dx)
    e = torch.exp(-g[:, 0].double().abs())
    want = e / (1 + e) ** 2 * float(dh[0, 0])
    assert_near(dx[:, 0], want, (2 * ROUND[dtype] + 2.0 ** -16) * want + 2 * TINY[dtype], "dg")


def test_sigmoid_slope_of_special_values():
    g = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), 200.0, -200.0, float("nan")])
    for dtype in DTYPES:
        t = TORCH[dtype]
        m = g.numel()
        one, zero, dx = torch.ones(1, 1, dtype=t).cuda(), torch.zeros(1, 1, dtype=t).cuda(), torch.empty(m, 1, dtype=t, device="cuda")
        ones = torch.ones(m, 1, dtype=t).cuda()
        with GatedPlan(m, 1, 1, dtype, "sigmoid") as plan:
            plan.backward(ones, ones, one, zero, g.to(t).view(m, 1).cuda(), ones, dX=dx)
        got = dx[:, 0].float().cpu().tolist()
        assert got[:6] == [0.25, 0.25, 0.0, 0.0, 0.0, 0.0] and got[6] != got[6]
