"""Sampling from 2^20 equal light logits beside a few heavy ones, in a batch whose rows
have one block each: a thread's share of the first, rough sum is then 4096 equal float32 terms,
whose roundings all go one way.  Top-p's cut lies among the heavy tokens, ever nearer to a
border of theirs; the last token that is kept comes out (the uniform number is the largest
below 1, and the heavy tokens lie in descending order).

Tolerance: a light weight is good to 2^-23 of itself, all of them together (under half of
the weight) to as much: cuts 2^-22 of the weight from a border are decided rightly."""

import math

import numpy as np
import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import SamplePlan
from layers_ref import TORCH

pytestmark = pytest.mark.gpu

VOCAB, ROWS = 2 ** 20, 640
#: the light tokens' logit: terms whose sums of 4096 are off by 2^-14 either way
LIGHT = [-11.625, -10.9375]


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
@pytest.mark.parametrize("z", LIGHT)
def test_cuts_next_to_a_border(z, dtype):
    heavy = 16
    row = np.full(VOCAB, z)
    places = np.arange(heavy) * 60001 + 17
    row[places] = -np.arange(heavy) / 32.0
    weights = np.exp(row[places])
    reach, total = np.cumsum(weights), math.fsum(weights) + (VOCAB - heavy) * math.exp(z)
    # 320 values of top_p on either side of the border behind the eighth token, 2^-22 ... 2^-13 of it away
    away = np.geomspace(2.0 ** -22, 2.0 ** -13, ROWS // 2)
    top_p = np.concatenate([reach[7] / total * (1 - away), reach[7] / total * (1 + away)]).astype(np.float32)
    targets = top_p.astype(np.float64) * total
    keep = np.abs(targets[:, None] - reach).min(1) / total > 2.0 ** -22
    assert keep.sum() > 0.75 * ROWS
    want = torch.from_numpy(places[np.searchsorted(reach, targets, side="left")])
    logits = torch.from_numpy(row).to(TORCH[dtype]).cuda().expand(ROWS, VOCAB).contiguous()
    p = torch.from_numpy(top_p).cuda()
    u = torch.full((ROWS,), 1 - 2.0 ** -24, device="cuda")

    def tokens(rows):
        out = torch.full((rows,), -77, dtype=torch.int64, device="cuda")
        with SamplePlan(rows, VOCAB, dtype) as plan:
            plan.forward(logits[:rows], u[:rows], out, top_p=p[:rows])
            torch.cuda.synchronize()
        return out.cpu()

    got = tokens(ROWS)
    assert torch.equal(got[torch.from_numpy(keep)], want[torch.from_numpy(keep)])
    for rows in (3, 100):                                    # with more blocks a row
        assert torch.equal(tokens(rows), got[:rows])
