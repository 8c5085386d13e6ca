"""Sampling at temperatures far below the distance of the element type's values near zero,
with the largest logit at zero (shifted logits, a saturated log softmax): for FLOAT16, whose
values are 2^-24 apart there, next to everything below the maximum then has no weight.

Tokens are equal and log probabilities as near as in test_sample_gpu.py."""

import pytest
import torch

from layers_ref import DTYPES, TORCH
from test_sample_gpu import check

pytestmark = pytest.mark.gpu

TEMPERATURES = [1e-7, 3e-8, 1.1e-8, 1e-9, 2e-10, 1.8e-10, 1e-12, 1e-15, 1e-25, 1e-30]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("settings", [{}, {"top_p": 0.9}, {"top_k": 5}, {"top_k": 400, "top_p": 0.8}, {"min_p": 0.01},
                                      {"min_p": 0.01, "top_p": 0.97}], ids=str)
@pytest.mark.parametrize("vocab", [300, 50257])
def test_the_maximum_at_zero(vocab, settings, dtype):
    rows = len(TEMPERATURES)
    gen = torch.Generator().manual_seed(vocab)
    logits = -torch.rand(rows, vocab, generator=gen) * 8 - 0.5
    # a few tokens within 2^-22 of the maximum, and two at it
    at = torch.randperm(vocab, generator=gen)[:11]
    logits[:, at[:9]] = -torch.arange(1.0, 10.0) * 2.0 ** -24
    logits[:, at[9:]] = 0.0
    u = torch.rand(rows, generator=gen)
    check(logits.to(TORCH[dtype]), u, dtype, temperature=torch.tensor(TEMPERATURES), **settings)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nothing_near_the_maximum(dtype):
    """Every uniform number gives the one token at zero, with probability one."""
    rows = len(TEMPERATURES)
    logits = torch.full((rows, 50257), -3.0)
    logits[torch.arange(rows), 777 + 4001 * torch.arange(rows)] = 0.0        # another place in every row
    check(logits.to(TORCH[dtype]), torch.linspace(0.01, 0.99, rows), dtype, temperature=torch.tensor(TEMPERATURES))
