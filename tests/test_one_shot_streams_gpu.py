"""The one-shot calls on another stream than torch's current one: their outputs
come from that stream's memory, never from a block that work queued on the
current stream still uses.  (The caching allocator hands a freed block to the
stream that it was allocated on, so the address tells.)"""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import gated, gemm, layer_norm, matmul, token_log_probs

pytestmark = pytest.mark.gpu


def freed_blocks(*shapes, dtype=torch.float32):
    """Addresses of blocks of these shapes, just freed by the current stream."""
    blocks = [torch.empty(s, dtype=dtype, device="cuda") for s in shapes for _ in range(4)]
    return {b.data_ptr() for b in blocks}


CALLS = {
    "matmul": lambda a, s: matmul(a, a, stream=s),
    "gemm": lambda a, s: gemm(a, a, stream=s),
    "layer_norm": lambda a, s: layer_norm(a, stream=s),
    "gated": lambda a, s: gated(a, a, a, stream=s),
    "token_log_probs": lambda a, s: token_log_probs(a, torch.zeros(a.shape[0], dtype=torch.int64, device="cuda"), top=3, stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
@pytest.mark.parametrize("handle", [False, True])
def test_outputs_are_memory_of_the_stream_that_writes_them(name, handle):
    n = 640
    a = torch.randn(n, n, device="cuda")
    want = CALLS[name](a, None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    seen = freed_blocks((n, n), (n,), (n, 3)) | freed_blocks((n, 3), dtype=torch.int64)
    got = CALLS[name](a, side.cuda_stream if handle else side)
    side.synchronize()
    for g, w in zip(*((v if isinstance(v, tuple) else (v,)) for v in (got, want))):
        assert torch.equal(g, w)
        assert g.data_ptr() not in seen, "a block of the current stream"


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gated_of_no_inputs_keeps_its_leading_dimensions(dtype):
    for lead in ((2, 3), (4,), (0, 5), ()):
        for trans_w in (False, True):
            x = torch.empty(lead + (0,), dtype=dtype, device="cuda")
            w = torch.empty((7, 0) if trans_w else (0, 7), dtype=dtype, device="cuda")
            h = gated(x, w, w, trans_w=trans_w)
            assert h.shape == lead + (7,) and not h.any()
