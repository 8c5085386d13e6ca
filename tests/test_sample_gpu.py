"""Sampling on the GPU against the definition in 64 bits.

Tokens have to be equal: a weight is good to 2^-36 of the largest, so that a choice
differs only where the uniform number or top_p lies that near to a border, which no
given input here does (the reference says how near it came, and the tests refuse inputs
below 2^-32).  Log probabilities: float32 weights' sums to 2^-34, and a logarithm of
float32, so 4 roundings of 1 and of the result."""

import math

import numpy as np
import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import OlcError, SamplePlan, sample
from layers_ref import DTYPES, F32, TORCH, Guarded

pytestmark = pytest.mark.gpu


def reference(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """token, log probability, the nearest border in shares of the weight."""
    z = np.asarray(z, np.float64)
    vocab = len(z)
    setting = (temperature, top_p, min_p, u)
    if np.isnan(z).any() or np.isposinf(z).any() or np.isnan(setting).any() or temperature < 0 or math.isinf(temperature):
        return -1, float("nan"), 1.0
    if np.isneginf(z).all():
        return -1, -float("inf"), 1.0
    order = np.argsort(-z, kind="stable")
    if temperature == 0:
        return int(order[0]), 0.0, 1.0
    w = np.exp((z - z.max()) / min(max(temperature, 2.0 ** -96), 2.0 ** 96))
    near = 1.0
    kept = order[:top_k] if 0 < top_k < vocab else order
    if top_p < 1:
        reach = np.cumsum(w[kept])
        target = float(np.float32(top_p)) * reach[-1]
        at = int(np.searchsorted(reach, target, side="left")) if top_p > 0 else 0
        if top_p > 0:
            near = min(near, np.abs(reach - target).min() / reach[-1])
        kept = kept[:at + 1]
    keep = w[kept] >= float(np.float32(min_p))
    keep[0] = True
    kept = np.sort(kept[keep])
    reach = np.cumsum(w[kept])
    target = min(max(float(np.float32(u)), 0.0), 1 - 2.0 ** -24) * reach[-1]
    at = int(np.searchsorted(reach, target, side="right"))
    if 0 < u < 1:
        near = min(near, np.abs(reach - target).min() / reach[-1])
    return int(kept[at]), math.log(w[kept[at]] / reach[-1]), near


def run(logits, u, dtype, pitch=None, offset=0, **settings):
    rows, vocab = logits.shape
    g = Guarded(rows, vocab, dtype, pitch, offset, logits)
    kinds = {"temperature": torch.float32, "top_k": torch.int32, "top_p": torch.float32, "min_p": torch.float32}
    given = {k: torch.as_tensor(v).to(kinds[k]).expand(rows).contiguous().cuda() for k, v in settings.items()}
    tokens, logprob = torch.full((rows + 8,), -77, dtype=torch.int64, device="cuda"), Guarded(1, rows, "float32")
    with SamplePlan(rows, vocab, dtype) as plan:
        plan.forward(g.t, u.float().cuda(), tokens[:rows], logprob=logprob.t.view(-1), **given)
        torch.cuda.synchronize()
    for x in (g, logprob):
        x.check_guards()
    assert (tokens[rows:] == -77).all()
    return tokens[:rows].cpu(), logprob.t.view(-1).cpu()


def check(logits, u, dtype, near=2.0 ** -32, **kw):
    tokens, logprob = run(logits, u, dtype, **kw)
    settings = {k: v for k, v in kw.items() if k not in ("pitch", "offset")}
    for r in range(len(u)):
        own = {k: (v[r].item() if torch.is_tensor(v) and v.dim() else float(v)) for k, v in settings.items()}
        if "top_k" in own:
            own["top_k"] = int(own["top_k"])
        for k in ("temperature", "top_p", "min_p"):
            if k in own:
                own[k] = float(np.float32(own[k]))
        token, lp, border = reference(logits[r].double().numpy(), float(u[r].float()), **own)
        assert border > near, "the input of row %d lies on a border" % r
        assert int(tokens[r]) == token, (r, own)
        if math.isnan(lp) or math.isinf(lp):
            assert str(float(logprob[r])) == str(lp), r
        else:
            assert abs(float(logprob[r]) - lp) <= 4 * F32 * (1 + abs(lp)), (r, float(logprob[r]), lp)


def draw(rows, vocab, dtype, seed, likely=20):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(rows, vocab, generator=g) * 2
    for r in range(rows):
        at = torch.randperm(vocab, generator=g)[:min(likely, vocab)]
        z[r, at] = torch.randn(len(at), generator=g) * 2.5 + 8
    return z.to(TORCH[dtype]), torch.rand(rows, generator=g)


def mixed(rows, vocab, seed):
    g = torch.Generator().manual_seed(seed)
    s = {"temperature": torch.rand(rows, generator=g) + 0.4, "top_k": torch.randint(0, min(vocab, 300), (rows,), generator=g),
         "top_p": torch.rand(rows, generator=g) * 0.5 + 0.6, "min_p": torch.rand(rows, generator=g) * 0.1}
    s["temperature"][::7] = 0
    s["min_p"][::3] = 0
    s["top_k"][::5] = 0
    s["top_p"][::4] = 1
    return s


VOCABS = [1, 2, 7, 33, 1000, 4099, 50257, 131072]
FILTERS = [{}, {"top_k": 50}, {"top_p": 0.9}, {"min_p": 0.02}, {"top_k": 3000}, {"top_k": 40, "top_p": 0.8},
           {"top_k": 5000, "top_p": 0.97, "min_p": 0.001}, "mixed"]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", VOCABS)
@pytest.mark.parametrize("which", range(len(FILTERS)))
def test_filters(which, vocab, dtype):
    rows = 24 if vocab < 10000 else 10
    logits, u = draw(rows, vocab, dtype, 100 * which + vocab)
    settings = mixed(rows, vocab, which) if FILTERS[which] == "mixed" else dict(FILTERS[which])
    settings.setdefault("temperature", torch.rand(rows, generator=torch.Generator().manual_seed(which)) + 0.5)
    check(logits, u, dtype, **settings)


@pytest.mark.parametrize("rows", [1, 2, 5, 40, 80, 160, 320])
def test_rows_of_every_cluster(rows):
    logits, u = draw(rows, 20011, "bfloat16", rows)
    check(logits, u, "bfloat16", **mixed(rows, 20011, rows))


def test_results_do_not_depend_on_the_cluster():
    logits, u = draw(700, 16384, "float16", 3)
    s = mixed(700, 16384, 4)
    many = run(logits, u, "float16", **s)
    for r in range(0, 700, 99):
        one = run(logits[r:r + 1], u[r:r + 1], "float16", **{k: v[r:r + 1] for k, v in s.items()})
        assert int(one[0]) == int(many[0][r]) and torch.equal(one[1], many[1][r:r + 1])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pitch,offset", [(1008, 0), (1003, 0), (1008, 1), (1005, 5)])
def test_pitches_and_offsets(pitch, offset, dtype):
    logits, u = draw(12, 1001, dtype, pitch)
    check(logits, u, dtype, pitch=pitch, offset=offset, top_p=0.95, temperature=0.9)
    check(logits, u, dtype, pitch=pitch, offset=offset, top_k=7)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [3, 1000, 5000, 70000])
def test_equal_logits(vocab, dtype):
    """Weights of one: the first ceil(top_p vocab) or top_k indices, each as likely."""
    u = torch.tensor([0.0, 0.1, 0.37, 0.5, 0.75, 0.9990234375])
    z = torch.full((6, vocab), 1.5).to(TORCH[dtype])
    for settings, kept in [({}, vocab), ({"top_p": 0.5}, math.ceil(vocab * 0.5)), ({"top_p": 0.8125}, math.ceil(vocab * 0.8125)),
                           ({"top_k": max(1, vocab - 300)}, max(1, vocab - 300)), ({"min_p": 1.0}, vocab),
                           ({"top_k": 2, "top_p": 0.75}, 2), ({"top_p": 0.0}, 1), ({"min_p": 2.0}, 1)]:
        tokens, logprob = run(z, u, dtype, **settings)
        want = torch.tensor([math.floor(float(v) * kept) for v in u])
        assert torch.equal(tokens, want), settings
        assert torch.allclose(logprob, torch.full((6,), -math.log(kept)), atol=4 * F32 * (1 + math.log(kept)), rtol=0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_equal_logits_below_others(dtype):
    """A step of equal logits that no list holds, cut by weight and by count."""
    vocab = 30000
    z = torch.full((8, vocab), 0.0)
    z[:, 1000:1004] = 6.0
    z[:, 20000:] = -40.0
    u = torch.rand(8, generator=torch.Generator().manual_seed(5))
    for s in ({"top_p": 0.9}, {"top_k": 9000}, {"top_k": 9000, "top_p": 0.9}, {"min_p": 0.002, "top_p": 0.99}):
        check(z.to(TORCH[dtype]), u, dtype, **s)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [100, 40000])
def test_masks(vocab, dtype):
    """Forbidden tokens: -inf, the type's lowest value, a row with one left, a row with none."""
    logits, u = draw(9, vocab, dtype, 9)
    low = torch.finfo(TORCH[dtype]).min
    half = torch.arange(vocab) % 2 == 0
    logits[0, half] = -math.inf
    logits[1, half] = low
    logits[2] = -math.inf
    logits[3] = -math.inf
    logits[3, vocab - 1] = -3.0
    logits[4] = low
    logits[5] = low
    logits[5, 5] = 0
    logits[6, 7] = math.inf
    logits[7, 3] = math.nan
    logits[8] = -math.inf
    logits[8, 4:40] = 1.0
    for s in ({}, {"top_k": 20}, {"top_p": 0.9}, {"min_p": 0.1}, {"temperature": 0.0}, {"top_k": 60, "top_p": 0.9}):
        check(logits, u, dtype, **s)


def test_strange_settings():
    logits, _ = draw(20, 500, "float32", 11)
    nan, inf = math.nan, math.inf
    t = torch.tensor([1.0, 1, 1, 1, nan, -1, inf, 1e-30, 1e30, 1e-45, 3e38, 1, 1, 1, 1, 1, 1, 1, 1, 1])
    p = torch.tensor([nan, 1, 1, 1, 1, 1, 1, 1, 1, 1, 1, -1, 0, 2, inf, 1e-30, 1e-45, 0.99999994, 0.5, 0.5])
    m = torch.tensor([0, nan, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, -1, 3])
    u = torch.tensor([0.5, 0.5, nan, 0.25, 0.5, 0.5, 0.5, 0.5, 0.53, 0.5, 0.51, 0.5, 0.5, -1, 1.5, inf, 0.3, 0.2, 1.0, 0.0])
    k = torch.tensor([0, 0, 0, -7, 0, 0, 0, 0, 0, 0, 0, 0, 0, 2 ** 31 - 1, 500, 501, 0, 499, -2 ** 31, 1])
    check(logits, u, "float32", near=2.0 ** -40, temperature=t, top_p=p, min_p=m, top_k=k)


@pytest.mark.parametrize("shift", [0.0, 1e4, -3e4, 1e30])
def test_logits_far_from_zero(shift):
    logits, u = draw(16, 3000, "float32", 13)
    logits = logits * (1.0 if abs(shift) < 1e20 else 1e25) + shift
    check(logits, u, "float32", top_p=0.9, temperature=1.0 if abs(shift) < 1e20 else 1e25)


@pytest.mark.parametrize("scale", [0.0, 1e-3, 0.3, 30.0])
def test_flat_and_steep_rows(scale):
    g = torch.Generator().manual_seed(17)
    logits = torch.randn(12, 30011, generator=g) * scale
    u = torch.rand(12, generator=g)
    for s in ({}, {"top_p": 0.37}, {"top_k": 11000, "top_p": 0.9}, {"min_p": 0.4}):
        if scale or "top_p" not in s:
            check(logits, u, "float32", near=2.0 ** -36, **s)


def test_frequencies():
    """Many uniform numbers on one row: each token as often as it is likely (a standard
    deviation of sqrt(n p (1 - p)); six of them for the worst of 40)."""
    n = 20000
    row = torch.randn(40, generator=torch.Generator().manual_seed(1)) * 1.5
    u = (torch.arange(n) + 0.5) / n
    tokens, _ = run(row.expand(n, 40).contiguous(), u, "float32", temperature=0.8)
    p = torch.softmax(row.double() / 0.8, 0)
    # evenly spaced numbers: off by at most one each way
    assert float((torch.bincount(tokens, minlength=40).double() - n * p).abs().max()) <= 1.01


def test_one_shot_graph_and_streams():
    logits, u = draw(33, 4099, "bfloat16", 19)
    want = run(logits, u, "bfloat16", temperature=0.7, top_k=30, top_p=0.9)
    g, gu = logits.cuda(), u.cuda()
    got = sample(g, gu, 0.7, 30, 0.9)
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])
    got = sample(g, gu, torch.full((33,), 0.7, device="cuda"), 30, 0.9)
    assert torch.equal(got[0].cpu(), want[0])
    with SamplePlan(33, 4099, "bfloat16") as plan:
        tokens = torch.empty(33, dtype=torch.int64, device="cuda")
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.forward(g, gu, tokens)
        gu.copy_(1 - gu)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(tokens, sample(g, gu)[0])


def test_refusals():
    with SamplePlan(4, 8, "float16") as plan:
        t = lambda *s, of=torch.float32: torch.zeros(s, dtype=of, device="cuda")  # noqa: E731
        z, u, tokens = t(4, 8, of=torch.float16), t(4), t(4, of=torch.int64)
        for args, kw in [((t(4, 9, of=torch.float16), u, tokens), {}), ((z, t(3), tokens), {}), ((z, u, tokens), {"top_p": t(5)}),
                         ((z.cpu(), u, tokens), {}), ((z, u, tokens), {"min_p": t(4).cpu()})]:
            with pytest.raises(ValueError):
                plan.forward(*args, **kw)
        for args, kw in [((z.float(), u, tokens), {}), ((z, u, tokens.int()), {}), ((z, u, tokens), {"top_k": t(4)}),
                         ((z, u.half(), tokens), {})]:
            with pytest.raises(TypeError):
                plan.forward(*args, **kw)
        lib, h = plan.lib, plan._h
        p = [x.data_ptr() for x in (z, u, tokens)]
        none = (None,) * 4
        assert lib.olc_sample_forward(h, p[0], 7, p[1], *none, p[2], None, None) == 13
        assert lib.olc_sample_forward(h, p[0] + 1, 8, p[1], *none, p[2], None, None) == 13
        assert lib.olc_sample_forward(h, p[0], 8, p[1], *none, p[2] + 4, None, None) == 13
        assert lib.olc_sample_forward(h, p[0], 8, None, *none, p[2], None, None) == 1
    with SamplePlan(0, 8, "float16") as plan:
        assert plan.lib.olc_sample_forward(plan._h, None, 8, None, *none, None, None, None) == 0
    for rows, vocab in [(4, 0), (4, 2 ** 20 + 1), (2 ** 27, 8)]:
        with pytest.raises(OlcError) as e:
            SamplePlan(rows, vocab, "float16")
        assert e.value.name == "OLC_ERR_INVALID"


@pytest.mark.parametrize("heat", [1.0, 3.0, 20.0, 300.0])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("top_p", [1.0, 0.7])
def test_a_flat_row_alone_and_among_others(top_p, dtype, heat):
    """Blocks of 1, 2 and 8 a row: the same token and the same bits of its log probability."""
    logits, u = draw(640, 20011, dtype, 71)
    of = lambda rows: run(logits[rows], u[rows], dtype, temperature=heat, top_p=top_p)  # noqa: E731
    tokens, logprob = of(slice(0, 640))
    for rows in (slice(0, 200), slice(0, 3), slice(100, 101), slice(630, 640)):
        some = of(rows)
        assert torch.equal(some[0], tokens[rows])
        assert torch.equal(some[1].view(torch.int32), logprob[rows].view(torch.int32))
