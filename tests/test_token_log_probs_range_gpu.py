"""Log probabilities of tokens over the whole range of their logits and
probabilities.  References and tolerances are those of the tests beside this
one."""

import pytest
import torch

from test_token_log_probs_gpu import check_backward

pytestmark = pytest.mark.gpu


def test_backward_keeps_the_smallest_probabilities():
    # p passes 2^-126 at log p = -87.3 and 0 at -103.3; p log p is a normal number for longer
    z = torch.linspace(0.0, -110.0, 4000).expand(3, 4000).contiguous()
    check_backward(3, 4000, "float32", z=z)
    check_backward(3, 4000, "float32", z=z, offset=1, d_offset=2)
