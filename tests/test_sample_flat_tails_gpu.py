"""Sampling of flat rows with a long tail of very light tokens, against the bound that the
header gives for them: with more than 512 tokens above 2^-12 of the largest weight a
lighter token's weight is good to 2^-23 of itself and 2^-32 of the largest.

`slack` below adds these up over the row: no sum of weights is off by more.  A token is right if
the uniform number's part of the whole falls into its share of the weight, give or take the slack
of both; so is a cut."""

import math

import numpy as np
import pytest
import torch

from layers_ref import DTYPES, F32, TORCH
from test_sample_gpu import run

pytestmark = pytest.mark.gpu


def row(vocab, top, tail, seed):
    """700 tokens within `top` octaves, the others `tail` octaves below the largest, give or take one."""
    g = np.random.default_rng(seed)
    x = -tail + g.uniform(-1, 1, vocab)
    places = g.permutation(vocab)[:700]
    x[places] = -g.uniform(0, top, 700)
    x[places[0]] = 0.0
    return x * math.log(2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,top,tail", [(20011, 1.4, 20), (20011, 2.8, 28), (300007, 1.4, 26), (300007, 11.0, 33), (300007, 1.4, 36)])
def test_tokens_of_the_tail(vocab, top, tail, dtype):
    z = torch.from_numpy(row(vocab, top, tail, vocab + tail)).to(TORCH[dtype])
    w = np.exp((z.double() - z.double().max()).numpy())
    light = w < 2.0 ** -12
    reach, total = np.cumsum(w), math.fsum(w)
    slack = float((w * 2.0 ** -23).sum()) + 2.0 ** -32 * vocab
    rows = 64
    g = np.random.default_rng(7)
    # half of the numbers fall on tokens of the tail
    u = np.concatenate([g.uniform(0, 1, rows // 2), (reach[g.choice(np.nonzero(light)[0], rows // 2)]) / total])
    u = np.minimum(u.astype(np.float32), np.float32(1 - 2.0 ** -24))
    logits = z.expand(rows, vocab).contiguous()
    tokens, logprob = run(logits, torch.from_numpy(u), dtype)
    t = tokens.numpy()
    assert ((0 <= t) & (t < vocab)).all()
    target = u.astype(np.float64) * total
    assert (reach[t] - w[t] - 2 * slack <= target).all() and (target <= reach[t] + 2 * slack).all()
    for r in range(rows):
        off = (w[t[r]] * 2.0 ** -23 + 2.0 ** -32) / w[t[r]] + slack / total
        if off < 0.25:
            lp = math.log(w[t[r]] / total)
            assert abs(float(logprob[r]) - lp) <= 2 * off + 4 * F32 * (1 + abs(lp)), r
    # the same of what top-p leaves: at least `few`, at most `many`
    order = np.argsort(-z.double().numpy(), kind="stable")
    sums = np.cumsum(w[order])
    rows = 12
    top_p = g.uniform(0.05, 0.999, rows).astype(np.float32)
    tokens, _ = run(logits[:rows], torch.full((rows,), 0.5), dtype, top_p=torch.from_numpy(top_p))
    for r in range(rows):
        aim = float(top_p[r]) * total
        few, many = (np.sort(order[:min(np.searchsorted(sums, aim + d), vocab - 1) + 1]) for d in (-2 * slack, 2 * slack))
        lowest = many[np.searchsorted(np.cumsum(w[many]), 0.5 * (w[few].sum() - slack) - slack, side="right")]
        above = np.searchsorted(np.cumsum(w[few]), 0.5 * (w[many].sum() + slack) + slack, side="right")
        highest = few[above] if above < len(few) else vocab - 1
        assert lowest <= int(tokens[r]) <= highest, r
