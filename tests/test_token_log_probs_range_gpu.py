"""Log probabilities of tokens over the whole range of their logits and
probabilities: finite masks of -1e9 and the like, rows of nothing else, logits
around large values, one token that holds everything, rows with an offset.
References and tolerances are those of the tests beside this one."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import TokenLogProbsPlan
from layers_ref import DTYPES, F32, TORCH, assert_near, normal
from test_token_log_probs_gpu import check_backward, check_forward, reference, rel_of, run_forward, tokens_of

pytestmark = pytest.mark.gpu


def test_backward_keeps_the_smallest_probabilities():
    # p passes 2^-126 at log p = -87.3 and 0 at -103.3; p log p is a normal number for longer
    z = torch.linspace(0.0, -110.0, 4000).expand(3, 4000).contiguous()
    check_backward(3, 4000, "float32", z=z)
    check_backward(3, 4000, "float32", z=z, offset=1, d_offset=2)


INF = float("inf")
#: finite masks and offsets; FLOAT16 reaches 65504
FAR = {"float32": [1e5, 1e9, 1e10, 1e12, 1e30, 1e37], "bfloat16": [1e5, 1e9, 1e10, 1e12, 1e30, 1e37],
       "float16": [1e4, 3e4, 49000.0, 5e4, 6e4]}


def far_rows(vocab, dtype, v, seed):
    t = TORCH[dtype]
    z = normal((14, vocab), dtype, seed, 3.0)
    z[0] = -v                                            # nothing but the mask
    z[1, :vocab // 2] = -v                               # whole slices of it
    few = z[2, [1, vocab // 3, vocab - 2]].clone()
    z[2] = -v                                            # three tokens left
    z[2, [1, vocab // 3, vocab - 2]] = few
    z[3, ::2] = -v
    z[4] = -v                                            # masks of both kinds and nothing else
    z[4, ::3] = -INF
    z[5, vocab // 2:] = -v                               # and beside what is left
    z[5, :vocab // 4] = -INF
    z[6, 3 * vocab // 4:] = -v
    z[7, vocab // 2] = v                                 # one token far above
    z[8, vocab // 2] = v                                 # the same, the rest masked
    z[8, :vocab // 2] = -INF
    z[8, vocab // 2 + 1:] = -v
    # neighbours of +-v in the type
    scale = float(torch.tensor(v, dtype=t)) * torch.finfo(t).eps
    z[9] = (normal((vocab,), "float32", seed + 1, 3.0).double() * min(scale, 1e300) + v).clamp(-float(torch.finfo(t).max), float(torch.finfo(t).max)).to(t)
    z[10] = -z[9]
    z[11] = -v
    z[11, vocab - 1] = float(torch.tensor(-v, dtype=t)) * (1 + 8 * torch.finfo(t).eps)
    # a ramp through the values where the sums change their unit
    ramp = torch.linspace(49000.0, 49300.0, vocab)
    z[12], z[13] = ramp.to(t), (-ramp).to(t)
    return z


@pytest.mark.parametrize("vocab", [600, 30000, 120000])
@pytest.mark.parametrize("dtype,v", [(d, v) for d in DTYPES for v in FAR[d]])
def test_finite_masks_and_far_logits(dtype, v, vocab):
    z = far_rows(vocab, dtype, v, 61)
    tokens = tokens_of(14, vocab, 62)
    tokens[2], tokens[5], tokens[8] = 1, vocab - 1, vocab // 2
    check_forward(z, tokens, dtype, 20)
    check_forward(z, tokens, dtype, 0, pitch=vocab + 3, offset=1)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("vocab", [700, 40000])
def test_maxima_that_move_far_within_a_row(vocab, dtype):
    # ascending and descending steps over many magnitudes, so that running maxima pass every unit
    z = torch.empty(4, vocab)
    steps = torch.tensor([-1e30, -1e10, -2e5, -49153.0, -49151.0, -40.0, 0.0, 40.0, 49151.0, 49153.0, 2e5, 1e10, 1e30])
    z[0] = steps[torch.arange(vocab) * 13 // vocab]
    z[1] = z[0].flip(0)
    z[2] = steps[:6][torch.arange(vocab) * 6 // vocab] + normal((vocab,), "float32", 63)
    z[3] = z[2].flip(0)
    z = z.to(TORCH[dtype])
    check_forward(z, tokens_of(4, vocab, 64), dtype, 5)


@pytest.mark.parametrize("same", [False, True])
@pytest.mark.parametrize("dtype,v", [(d, v) for d in DTYPES for v in FAR[d]])
def test_backward_of_finite_masks_and_far_logits(dtype, v, same):
    for vocab, kw in ((4000, {}), (4001, {"pitch": 4009, "offset": 3})):
        check_backward(14, vocab, dtype, z=far_rows(vocab, dtype, v, 65), same=same, **kw)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [300, 50257])
def test_a_single_token_left_has_all_of_the_probability(vocab, dtype):
    """logprob is log 1, and lse that token's logit: off by the sum's own
    error (one exponential of 1: 2^-21) and lse's one rounding, not by
    roundings of the logit's size."""
    rows = 200
    value = normal((rows,), dtype, 71, 300.0)
    tokens = tokens_of(rows, vocab, 72)
    for mask in (-INF, -30000.0):
        z = torch.full((rows, vocab), mask).to(TORCH[dtype])
        z[torch.arange(rows), tokens] = value
        logprob, entropy, lse, best, index = run_forward(z, tokens, dtype, 1)
        assert float(logprob.abs().max()) <= 2.0 ** -21
        assert float(best.abs().max()) <= 2.0 ** -21 and torch.equal(index[:, 0].cpu(), tokens)
        assert_near(lse, value.double(), 2.0 ** -21 + F32 * value.double().abs(), "lse")
        assert float(entropy.abs().max()) <= 2.0 ** -20


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [-900.0, 1500.0, 30000.0])
@pytest.mark.parametrize("rows,vocab", [(5, 700), (2, 60000), (400, 1003)])
def test_log_probabilities_do_not_depend_on_an_offset(rows, vocab, shift, dtype):
    """logprob = (z - m) - log s takes no rounding of lse's size: off by the
    sum's error and roundings of its own size alone."""
    z = normal((rows, vocab), dtype, 73, 3.0, shift)
    tokens = tokens_of(rows, vocab, 74)
    got = run_forward(z, tokens, dtype, 7)
    logprob, entropy, lse, best, order = reference(z, tokens, 7)
    rel = rel_of(vocab)
    assert_near(got[0], logprob, rel + 4 * F32 * logprob.abs(), "logprob")
    assert_near(got[3], best, rel + 4 * F32 * best.abs(), "alternatives' log probabilities")
    assert_near(got[2], lse, rel + F32 * lse.abs(), "lse")
    assert torch.equal(got[4].cpu(), order)
    d = torch.empty(rows, vocab, dtype=TORCH[dtype], device="cuda")
    one = torch.ones(rows, device="cuda")
    with TokenLogProbsPlan(rows, vocab, dtype) as plan:         # a gradient's entries add up to nothing
        plan.backward(z.cuda(), tokens.cuda(), lse.float().cuda(), None, one, d)
    assert float(d.double().sum(-1).abs().max()) <= 2.0 ** -7 * 2 + 4 * F32 * abs(shift) * 2


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shift", [0.0, 50.0, 300.0, -2000.0])
@pytest.mark.parametrize("rows,vocab", [(107, 18), (24, 880), (11, 16468), (3, 57298)])
def test_backward_of_peaked_rows_with_an_offset(rows, vocab, shift, dtype):
    # one token near certain, the rest down to the smallest probabilities: errors of log p's size, not of lse's
    z = normal((rows, vocab), dtype, 81, 20.0, shift)
    check_backward(rows, vocab, dtype, z=z)
    check_backward(rows, vocab, dtype, z=z, with_lp=False)
    check_backward(rows, vocab, dtype, z=z, offset=3, d_offset=1)


def test_backward_of_tiny_gradients():
    # dlogprob and dentropy near float32's smallest values keep their digits
    rows, vocab = 4, 500
    z = normal((rows, vocab), "float32", 82, 3.0)
    tokens = tokens_of(rows, vocab, 83).cuda()
    lse, entropy = (v.float().cuda() for v in (lambda r: (r[2], r[1]))(reference(z, tokens.cpu(), 0)))
    d, e = (torch.empty(rows, vocab, device="cuda") for _ in range(2))
    dlp, dh = normal((rows,), "float32", 84).cuda(), normal((rows,), "float32", 85).cuda()
    small = 2.0 ** -104
    with TokenLogProbsPlan(rows, vocab, "float32") as plan:
        plan.backward(z.cuda(), tokens, lse, entropy, dlp, d, dentropy=dh)
        plan.backward(z.cuda(), tokens, lse, entropy, dlp * small, e, dentropy=dh * small)
    # a few roundings of each term: p is off by 2^-21 + |log p| 2^-23 of itself, the bracket's terms by as much
    terms = (dlp.abs() + dh.abs() * 40)[:, None].double()
    assert ((e.double() / small - d.double()).abs() <= 2.0 ** -18 * terms).all()
    big = d.abs() > 2.0 ** -12
    assert ((e.double() / small / d.double())[big] - 1).abs().max() <= 2.0 ** -8 and int(big.sum()) > 100
