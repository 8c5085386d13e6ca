"""Plans whose calls come over the default streams of several host threads, and
over streams whose handles are used again, one call after the other on the host
but not on the GPU."""

import ctypes
import threading

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import GatedPlan, LayerNormPlan
from layers_ref import normal

pytestmark = pytest.mark.gpu

PER_THREAD = 2          # the handle of every host thread's own default stream


def in_thread(f):
    out = []
    t = threading.Thread(target=lambda: out.append(f()))
    t.start()
    t.join()
    return out[0]


def test_threads_default_streams_have_identities_of_their_own():
    torch.zeros(1, device="cuda")
    cuda = ctypes.CDLL("libcuda.so.1")
    device = torch.cuda.current_device()

    def identity():
        torch.cuda.set_device(device)
        torch.zeros(1, device="cuda")
        n = ctypes.c_ulonglong()
        assert cuda.cuStreamGetId(ctypes.c_void_p(PER_THREAD), ctypes.byref(n)) == 0
        return n.value

    assert len({identity(), in_thread(identity), identity(), in_thread(identity)}) == 3


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_one_plan_on_the_default_streams_of_threads(dtype):
    m, d, f = 200, 2048, 512
    x, wg, wu = (normal(s, dtype, i, 0.02).cuda() for i, s in enumerate([(m, d), (d, f), (d, f)]))
    g, u, dh = (normal((m, f), dtype, 5 + i).cuda() for i in range(3))
    norm_x = normal((m, d), dtype, 9).cuda()
    stats = [torch.zeros(m, device="cuda"), torch.ones(m, device="cuda")]
    with GatedPlan(m, d, f, dtype) as plan, LayerNormPlan(m, d, dtype) as norm:
        def step():
            out = [torch.empty_like(dh), torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu),
                   torch.empty_like(x), torch.empty(d, dtype=x.dtype, device="cuda")]
            torch.cuda.current_stream().synchronize()
            plan.forward(x, wg, wu, out[0], stream=PER_THREAD)
            plan.backward(dh, x, wg, wu, g, u, *out[1:4], stream=PER_THREAD)
            norm.backward(x, norm_x, None, *stats, out[4], dgamma=out[5], stream=PER_THREAD)
            return out

        want = step()
        torch.cuda.synchronize()
        got = [in_thread(step) for _ in range(8)]
        torch.cuda.synchronize()
        for o in got:
            assert all(torch.equal(a, b) for a, b in zip(o, want))
