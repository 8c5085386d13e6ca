"""The first call of a plan: a FLOAT plan has its counters from the start, so
that a call which needs no other memory can be the first one inside a capture."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import GatedPlan
from layers_ref import normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,d,f,trans_w", [(300, 64, 200, False), (5, 33, 70, False), (3, 48, 100, True)])
def test_a_float_plans_first_call_is_captured(m, d, f, trans_w):
    # a K of at most 7 slices of 16 is never cut into pieces: no partial sums
    x, wg, wu = (normal(s, "float32", i).cuda() for i, s in enumerate([(m, d)] + 2 * [(f, d) if trans_w else (d, f)]))
    want, got = torch.empty(m, f, device="cuda"), torch.zeros(m, f, device="cuda")
    with GatedPlan(m, d, f, "float32", "silu", trans_w) as plan:
        plan.forward(x, wg, wu, want)
    with GatedPlan(m, d, f, "float32", "silu", trans_w) as plan:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.forward(x, wg, wu, got)
        for _ in range(2):
            got.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
