"""The embedding, residual norm and sampling plans on streams: one plan over the
default streams of several host threads, outputs of the one-shot calls in the memory of
their stream, and a graph that outlives a later, larger call of its plan."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import EmbeddingPlan, ResidualNormPlan, SamplePlan, embedding, residual_norm, sample
from layers_ref import normal
from test_one_shot_streams_gpu import freed_blocks
from test_plan_streams_gpu import PER_THREAD, in_thread

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_one_plan_on_the_default_streams_of_threads(dtype):
    n, vocab, d = 3000, 700, 1024
    ids = torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(1)).cuda()
    dy, y, f = (normal((n, d), dtype, 2 + i).cuda() for i in range(3))
    stats = torch.ones(4, n, device="cuda")
    gamma = normal((d,), dtype, 9).cuda()
    with EmbeddingPlan(n, vocab, d, dtype) as embed, ResidualNormPlan(n, d, dtype, after=True) as join:
        def step():
            out = [torch.empty(vocab, d, dtype=dy.dtype, device="cuda"), torch.empty_like(dy), torch.empty_like(dy),
                   torch.empty_like(gamma), torch.empty_like(gamma)]
            torch.cuda.current_stream().synchronize()
            embed.backward(dy, ids, out[0], stream=PER_THREAD)
            join.backward(dy, f, f, y, stats, gamma=gamma, after_gamma=gamma, dX=out[1], dF=out[2], dgamma=out[3],
                          dafter_gamma=out[4], stream=PER_THREAD)
            return out

        want = step()
        torch.cuda.synchronize()
        got = [in_thread(step) for _ in range(8)]
        torch.cuda.synchronize()
        for o in got:
            assert all(torch.equal(a, b) for a, b in zip(o, want))


CALLS = {
    "embedding": lambda a, s: embedding(a, torch.arange(a.shape[0], device="cuda"), 2.0, stream=s),
    "residual_norm": lambda a, s: residual_norm(a, a, stream=s),
    "sample": lambda a, s: sample(a, torch.full((a.shape[0],), 0.5, device="cuda"), 0.8, 20, 0.9, 0.01, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_are_memory_of_the_stream_that_writes_them(name, handle):
    n = 640
    a = torch.randn(n, n, device="cuda")
    want = CALLS[name](a, None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    seen = freed_blocks((n, n), (n,)) | freed_blocks((n,), dtype=torch.int64)
    side.wait_stream(torch.cuda.current_stream())
    got = CALLS[name](a, side.cuda_stream if handle else side)
    side.synchronize()
    torch.cuda.synchronize()
    for g, w in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, want))):
        assert torch.equal(g, w)
        assert g.data_ptr() not in seen, "a block of the current stream"


def test_a_graph_keeps_its_memory_when_the_plan_takes_more():
    """Every call of a plan finds its memory made by the first one, whatever operands the
    later ones give: nothing is allocated while a stream captures."""
    n, vocab, d = 200, 90, 1032
    dy, f, y = (normal((n, d), "float16", i).cuda() for i in range(3))
    ids = torch.arange(n, device="cuda") % vocab
    odd = torch.empty(n * d + 1, dtype=torch.float16, device="cuda")[1:].view(n, d)
    odd.copy_(dy)
    stats = torch.ones(4, n, device="cuda")
    vectors = [torch.empty(d, dtype=torch.float16, device="cuda") for _ in range(5)]
    gate = torch.ones(d, dtype=torch.float16, device="cuda")
    with EmbeddingPlan(n, vocab, d, "float16") as embed, ResidualNormPlan(n, d, "float16", after=True) as join:
        de, dx = torch.empty(vocab, d, dtype=torch.float16, device="cuda"), torch.empty_like(dy)
        embed.backward(dy, ids, de)
        join.backward(dy, None, f, y, stats, dX=dx)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            embed.backward(odd, ids, de)
            join.backward(odd, f, f, y, stats, gate=gate, dX=dx, dF=odd, dgate=vectors[0], dgamma=vectors[1],
                          dbeta=vectors[2], dafter_gamma=vectors[3], dafter_beta=vectors[4])
        graph.replay()
        torch.cuda.synchronize()
        want = embed.backward(dy, ids, torch.empty_like(de))
        # other chunks of the sums, float32, and one rounding of either
        assert float((de.double() - want.double()).abs().max()) <= 2.0 ** -10 * float(want.abs().max())


def test_plans_of_one_size_do_not_share_memory():
    """Two plans' calls at once on two streams."""
    n, vocab, d = 4000, 50, 512
    ids = [torch.randint(0, vocab, (n,), generator=torch.Generator().manual_seed(i)).cuda() for i in range(2)]
    dy = normal((n, d), "float32", 3).cuda()
    plans = [EmbeddingPlan(n, vocab, d, "float32") for _ in range(2)]
    want = [plans[i].backward(dy, ids[i], torch.empty(vocab, d, device="cuda")) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [torch.empty(vocab, d, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            plans[i].backward(dy, ids[i], out[i], stream=streams[i])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_one_sampling_plan_on_two_streams_at_once():
    """It has no memory of its own."""
    z, u = normal((64, 9000), "bfloat16", 1, 3.0).cuda(), torch.rand(64, device="cuda")
    with SamplePlan(64, 9000, "bfloat16") as plan:
        want = plan.forward(z, u, torch.empty(64, dtype=torch.int64, device="cuda"))
        streams = [torch.cuda.Stream() for _ in range(2)]
        out = [torch.empty_like(want) for _ in range(2)]
        torch.cuda.synchronize()
        for _ in range(10):
            for o, s in zip(out, streams):
                plan.forward(z, u, o, stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in out)
