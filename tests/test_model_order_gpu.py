"""The token model's gradients belong to its last forward call: with other
activations in their place since then there are none."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300.model import TokenModel, parameters

pytestmark = pytest.mark.gpu


def test_gradients_after_something_else():
    rows, vocab = 24, 200
    p = parameters(1, 64, 96, vocab, "float32", seed=2)
    model = TokenModel(rows, 1, 64, 96, vocab, "float32")
    gen = torch.Generator().manual_seed(1)
    ids, targets, others = (torch.randint(0, vocab, (rows,), generator=gen).cuda() for _ in range(3))
    dlp, u = torch.full((rows,), 1.0 / rows, device="cuda"), torch.rand(rows, generator=gen).cuda()
    with pytest.raises(RuntimeError):
        model.backward(dlp)                                  # no forward call at all
    model.forward(ids, targets, p)
    want = model.backward(dlp)
    again = model.backward(dlp)                              # as often as one likes
    assert all(torch.equal(again[k], want[k]) for k in want)
    for other in (lambda: model.next_tokens(others, u, p), lambda: model.logits(others, p)):
        model.forward(ids, targets, p)
        other()
        with pytest.raises(RuntimeError):
            model.backward(dlp)
        model.forward(ids, targets, p)
        got = model.backward(dlp)
        assert all(torch.equal(got[k], want[k]) for k in want)
