"""The first call of a plan can be the one that is captured: what every forward
call needs is there when the plan is."""

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


@pytest.mark.parametrize("dtype,m,d,f", [("float32", 70, 2000, 100), ("float32", 1030, 300, 3000), ("float32", 2, 96, 64),
                                         ("float32", 1, 1000, 2730), ("bfloat16", 200, 4096, 512), ("float16", 128, 4096, 1024)])
def test_a_forward_call_needs_no_memory_after_creation(dtype, m, d, f):
    # partial sums, K slices and what is not kept: all there when the plan is (rows on 16-byte boundaries)
    x, wg, wu = (normal(s, dtype, i, 0.05).cuda() for i, s in enumerate([(m, d), (d, f), (d, f)]))
    want, got = (torch.zeros(m, f, dtype=x.dtype, device="cuda") for _ in range(2))
    with GatedPlan(m, d, f, dtype) as plan:
        plan.forward(x, wg, wu, want)
        torch.cuda.synchronize()
    with GatedPlan(m, d, f, dtype) as plan:
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.forward(x, wg, wu, got)
        for _ in range(2):
            got.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(got, want)
        h = torch.empty_like(want)
        plan.forward(x, wg, wu, h)
        torch.cuda.synchronize()
        assert torch.equal(h, want)
