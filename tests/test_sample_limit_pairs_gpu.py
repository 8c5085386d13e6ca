"""Sampling of rows with many equal light tokens just below the limit of the heavy ones.

A token is light when the rounded (z - m) log2(e) / T is the float32 next below -12 (-6
and -3 in flat rows), and its weight can still round up to 2^31, the limit's own: a sum of
two of them does not fit 32 bits.  The values here were found by forming such weights
in float32 on a CPU.

Tolerances: a light weight is good to 2^-23 of itself, so sums of them to as much; the
uniform numbers stay 2^-22 of the whole weight from every border.  The log probability has that
and four float32 roundings of 1 and of itself."""

import math

import numpy as np
import pytest
import torch

from layers_ref import F32, TORCH
from test_sample_gpu import reference, run

pytestmark = pytest.mark.gpu

#: element type, temperature, the maximum, the light tokens' logit
PLAIN = [("bfloat16", 1.19573712, 9.9375, -0.00836181641), ("bfloat16", 1.19567108, 8.5625, -1.3828125),
         ("bfloat16", 1.15116656, 9.5625, -0.0126342773), ("bfloat16", 0.323103577, 11.875, 9.1875),
         ("float16", 0.323103577, -8.53125, -11.21875), ("float16", 1.42719734, 11.875, 0.00390625),
         ("float32", 0.612005651, 5.09051991, 0.0), ("float32", 1.31416976, 10.9309568, 0.0)]
#: and the limit, -6 or -3 octaves from the maximum
FLAT = [("bfloat16", 0.683777332, -3.75, -6.59375, 6), ("bfloat16", 0.646207154, 10.8125, 8.125, 6),
        ("bfloat16", 1.38821828, -0.67578125, -3.5625, 3), ("bfloat16", 2.69002509, -1.0625, -6.65625, 3),
        ("float16", 1.24545157, 2.84960938, -2.33007812, 6), ("float16", 2.54584956, 0.439453125, -10.1484375, 6),
        ("float16", 1.88132691, -1.77929688, -5.69140625, 3), ("float32", 2.10395479, 8.75010204, 0.0, 6),
        ("float32", 0.612005651, 1.27262998, 0.0, 3)]


def check(z, dtype, temperature, offset, **settings):
    """Evenly spaced uniform numbers; the row starts `offset` elements behind a 16-byte boundary."""
    rows = 24
    logits = torch.tensor(z, dtype=torch.float64).to(TORCH[dtype]).expand(rows, len(z)).contiguous()
    assert torch.equal(logits[0].double(), torch.tensor(z, dtype=torch.float32).double())    # nothing was rounded
    u = (torch.arange(rows) + 0.4363) / rows
    tokens, logprob = run(logits, u, dtype, pitch=len(z) + 16, offset=offset, temperature=temperature, **settings)
    for r in range(rows):
        token, lp, border = reference(logits[r].double().numpy(), float(u[r]), float(np.float32(temperature)), **settings)
        assert border > 2.0 ** -22, "the input of row %d lies on a border" % r
        assert int(tokens[r]) == token, r
        assert abs(float(logprob[r]) - lp) <= 2 * F32 + 4 * F32 * (1 + abs(lp)), r


def row(dtype, m, z, vocab):
    v = np.full(vocab, np.float32(z))
    v[0] = np.float32(m)
    return v


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("settings", [{}, {"top_p": 0.999}], ids=["all", "top_p"])
@pytest.mark.parametrize("dtype,temperature,m,z", PLAIN)
def test_equal_tokens_below_the_limit(dtype, temperature, m, z, settings, offset):
    check(row(dtype, m, z, 1000), dtype, temperature, offset, **settings)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("dtype,temperature,m,z,octaves", FLAT)
def test_equal_tokens_below_the_limit_of_a_flat_row(dtype, temperature, m, z, octaves, offset):
    """400 tokens at the maximum, and 4000 just below the limit, where more than 512 would be heavy."""
    assert abs((m - z) / temperature / math.log(2) - octaves) < 1e-5
    v = row(dtype, m, z, 4400)
    v[4000:] = np.float32(m)
    check(v, dtype, temperature, offset)
