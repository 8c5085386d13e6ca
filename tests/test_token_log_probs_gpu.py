"""Log probabilities of tokens on the GPU, with entropy and alternatives, and
their gradient, against the definition in 64 bits.

Tolerances.  Each exponential is good to 2^-21 of itself plus |d| 2^-23 for
its argument d (rounded once after the scaling by log2 e); elements with
|d| > 32 weigh less than 2^-46.  A sum of positive terms over a chain of DEPTH
additions is off by DEPTH 2^-24 of itself.  So s is off by at most
REL = 2^-21 + 32 * 2^-23 + DEPTH * 2^-24 relatively, and so is a; DEPTH is a
thread's own elements plus its joins, 800 for the longest row here.  lse =
m + log s adds the rounding of m + log s itself.  Integers have to be equal."""

import math

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import OlcError, TokenLogProbsPlan, token_log_probs
from layers_ref import DTYPES, F32, ROUND, TINY, TORCH, Guarded, assert_near, normal

pytestmark = pytest.mark.gpu

INF = math.inf


def rel_of(vocab):
    return 2.0 ** -21 + 32 * 2.0 ** -23 + (vocab / 512 + 64) * F32


def reference(z, tokens, top):
    z = z.double()
    m = z.amax(-1, keepdim=True)
    r = torch.where(m == -INF, 0.0, m)
    e = torch.exp(z - r)
    s = e.sum(-1)
    nothing = s == 0
    d = torch.where(e > 0, z - r, 0.0)
    lse = torch.where(nothing, -INF, r[:, 0] + torch.log(s))
    entropy = torch.where(nothing, 0.0, torch.log(s) - (d * e).sum(-1) / s)
    at = z.gather(1, tokens.clamp(0, z.shape[1] - 1)[:, None])[:, 0]
    logprob = torch.where(nothing, -INF, at - lse)
    logprob = torch.where(tokens < 0, 0.0, torch.where(tokens >= z.shape[1], math.nan, logprob))
    order = torch.sort(z, dim=-1, descending=True, stable=True).indices[:, :top]
    best = torch.where(nothing[:, None], -INF, z.gather(1, order) - lse[:, None])
    return logprob, entropy, lse, best, order


def run_forward(z, tokens, dtype, top, pitch=None, offset=0):
    rows, vocab = z.shape
    g = Guarded(rows, vocab, dtype, pitch, offset, z)
    lp, en, ls = (Guarded(1, rows, "float32") for _ in range(3))
    best = Guarded(1, rows * top, "float32")
    index = torch.full((rows * top + 8,), -77, dtype=torch.int64, device="cuda")
    with TokenLogProbsPlan(rows, vocab, dtype, top) as plan:
        plan.forward(g.t, tokens.cuda(), lp.t[0], entropy=en.t[0], lse=ls.t[0],
                     top_logprob=best.t[0] if top else None, top_index=index[:rows * top] if top else None)
        torch.cuda.synchronize()
    for x in (g, lp, en, ls, best):
        x.check_guards()
    assert (index[rows * top:] == -77).all()
    return lp.t[0], en.t[0], ls.t[0], best.t.view(rows, top), index[:rows * top].view(rows, top)


def check_forward(z, tokens, dtype, top, **kw):
    got = run_forward(z, tokens, dtype, top, **kw)
    logprob, entropy, lse, best, order = reference(z, tokens, top)
    rel = rel_of(z.shape[1])
    fine = torch.where(torch.isfinite(lse), lse.abs(), 0.0)
    off = rel + 4 * F32 * fine
    assert_near(got[2], lse, off, "lse")
    assert_near(got[0], logprob, off + 4 * F32 * logprob.abs().nan_to_num(0, 0, 0), "logprob")
    # both terms are positive, log s is off by rel and a / s by twice that
    assert_near(got[1], entropy, rel * (1 + 2 * entropy) + 4 * F32 * entropy, "entropy")
    assert torch.equal(got[4].cpu(), order), "alternatives"
    assert_near(got[3], best, off[:, None] + 4 * F32 * best.abs().nan_to_num(0, 0, 0), "their log probabilities")


def tokens_of(rows, vocab, seed):
    return torch.randint(0, vocab, (rows,), generator=torch.Generator().manual_seed(seed))


SIZES = [(1, 1, 1), (5, 2, 2), (3, 7, 7), (4, 33, 5), (700, 100, 20), (9, 4097, 32), (3, 50257, 20), (400, 5003, 5),
         (1, 200000, 32), (40, 16384, 1), (2, 65536, 0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,top", SIZES)
def test_forward(rows, vocab, top, dtype):
    check_forward(normal((rows, vocab), dtype, 1, 3.0), tokens_of(rows, vocab, 2), dtype, top)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,pitch,offset", [(1000, 1008, 0), (1000, 1001, 0), (1001, 1001, 3), (20011, 20016, 8), (3, 9, 1)])
def test_forward_pitches_and_offsets(vocab, pitch, offset, dtype):
    check_forward(normal((11, vocab), dtype, 3, 3.0), tokens_of(11, vocab, 4), dtype, min(vocab, 7), pitch=pitch, offset=offset)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab", [600, 30000, 120000])
def test_masks(vocab, dtype):
    low = torch.finfo(TORCH[dtype]).min
    z = normal((12, vocab), dtype, 5, 3.0)
    z[0] = -INF                                   # nothing left
    z[1] = low                                    # the lowest value everywhere: a uniform row
    z[2, 1:] = -INF                               # one token left
    z[3, 3:vocab - 3] = -INF                      # fewer than the alternatives asked for
    z[4, : vocab // 2] = -INF                     # a whole slice masked
    z[5, vocab // 2:] = low
    z[6, ::2] = -INF
    z[7, :] = -INF
    z[7, vocab - 1] = low                         # a single lowest value
    z[8] = 1.5                                    # every value equal
    z[9, 5] = torch.finfo(TORCH[dtype]).max       # finite, and far above
    z[10] = 0.0
    z[10, 1::2] = -0.0                            # zeros of both signs are equal
    tokens = tokens_of(12, vocab, 6)
    tokens[2], tokens[3], tokens[6] = 5, vocab - 1, 2     # masked ones among them
    check_forward(z, tokens, dtype, 20)


@pytest.mark.parametrize("vocab", [3000, 70000])
def test_alternatives_where_few_threads_hold_the_largest(vocab):
    # the largest values packed into what one thread, four neighbours or one block's tail reads, and ramps
    z = torch.zeros(6, vocab)
    z[0, 1024:2048] = torch.arange(1024.0)
    z[1] = torch.arange(float(vocab))
    z[2] = -torch.arange(float(vocab))
    for j in range(0, vocab - 8, 2048):
        z[3, j:j + 8] = torch.arange(8.0) + j
    z[4, -5:] = torch.tensor([3.0, 9.0, 9.0, 1.0, 9.0])
    # more elements above the bound than the buffer holds: all of one group's packs
    for j in range(0, vocab - 32, 4096):
        z[5, j:j + 32] = 1.0 + torch.rand(32, generator=torch.Generator().manual_seed(j))
    for top in (1, 20, 32):
        check_forward(z * 2.0 ** -8, tokens_of(6, vocab, 8), "float32", top)


def test_more_above_the_bound_than_the_buffer_holds():
    # four neighbouring threads hold the 3000 largest values: the bound is a value far below them
    vocab = 400000
    z = torch.zeros(400, vocab, dtype=torch.bfloat16)
    z[:, :] = -5.0
    i = torch.arange(vocab)
    mine = ((i // 8) % 512) < 4
    z[:, mine] = (1.0 + (torch.arange(int(mine.sum())) % 97) / 64).bfloat16()
    tokens = tokens_of(400, vocab, 9)
    got = run_forward(z, tokens, "bfloat16", 32)
    _, _, _, _, order = reference(z[:1], tokens[:1], 32)
    assert torch.equal(got[4].cpu(), order.expand(400, 32))


@pytest.mark.parametrize("vocab", [500, 40000])
def test_special_values_and_tokens(vocab):
    z = normal((8, vocab), "float32", 10, 3.0)
    z[1, 7] = math.nan
    z[2, 9] = INF
    z[3, :] = math.nan
    z[5, 11] = math.nan
    z[5, 12] = -INF
    tokens = tokens_of(8, vocab, 11)
    tokens[4], tokens[6], tokens[7] = -1, vocab, 2 ** 40
    lp, en, ls, best, index = (v.cpu() for v in run_forward(z, tokens, "float32", 3))
    for r in (1, 2, 3, 5):
        assert torch.isnan(lp[r]) and torch.isnan(en[r]) and torch.isnan(ls[r]), r
    assert int(index[1, 0]) == 7 and int(index[2, 0]) == 9 and int(index[5, 0]) == 11
    assert index[3].tolist() == [0, 1, 2]
    rest = [1, 2, 3, 4]
    fine = z[1].clone()
    fine[7] = -INF
    assert index[1, 1:].tolist() == torch.sort(fine, descending=True, stable=True).indices[:2].tolist(), rest
    assert float(lp[4]) == 0.0 and torch.isnan(lp[6]) and torch.isnan(lp[7])
    ok = [0, 4, 6, 7]
    want = reference(z[ok], tokens[ok], 3)
    assert torch.equal(index[ok], want[4])
    assert_near(ls[ok], want[2], 2 * rel_of(vocab) + 4 * F32 * want[2].abs(), "lse")


# ---- backward ------------------------------------------------------------------


def reference_grad(z, tokens, lse, entropy, dlp, dh):
    z, lse = z.double(), lse.double()[:, None]
    rows, vocab = z.shape
    nothing = lse == -INF
    logp = z - torch.where(nothing, 0.0, lse)
    p = torch.exp(logp)
    d = torch.zeros_like(z) if dlp is None else torch.where(tokens < 0, 0.0, dlp.double())[:, None].expand(rows, vocab)
    h = torch.zeros_like(z) if dh is None else dh.double()[:, None].expand(rows, vocab)
    e = torch.zeros(rows, 1, dtype=torch.float64) if dh is None else entropy.double()[:, None]
    inner = torch.where(p > 0, d + h * (logp + e), 0.0)
    g = -p * inner
    hit = torch.arange(vocab)[None] == tokens[:, None]
    g = torch.where(hit, g + d, g)
    # p is off by 2^-21 + |log p| 2^-23 of itself and by lse's rounding; the bracket and the products a few roundings
    seen = torch.where(p > 0, logp.abs(), 0.0)
    off = p * (d.abs() + h.abs() * (seen + e.abs())) * (2.0 ** -21 + (seen + 8) * 2.0 ** -23 + torch.where(nothing, 0.0, lse.abs()) * 4 * F32)
    off = off + 4 * F32 * torch.where(hit, d.abs(), 0.0)
    return torch.where(nothing, 0.0, g), torch.where(nothing, 0.0, off)


def check_backward(rows, vocab, dtype, pitch=None, offset=0, d_offset=None, with_lp=True, with_h=True, same=False, z=None):
    z = normal((rows, vocab), dtype, 21, 3.0) if z is None else z
    tokens = tokens_of(rows, vocab, 22)
    if rows > 4:
        tokens[3] = -100
    _, entropy, lse, _, _ = reference(z, tokens, 0)
    entropy, lse = entropy.float(), lse.float()
    dlp, dh = normal((rows,), "float32", 23) if with_lp else None, normal((rows,), "float32", 24) if with_h else None
    gz = Guarded(rows, vocab, dtype, pitch, offset, z)
    gd = gz if same else Guarded(rows, vocab, dtype, pitch, offset if d_offset is None else d_offset)
    up = lambda t: None if t is None else t.cuda()  # noqa: E731
    with TokenLogProbsPlan(rows, vocab, dtype) as plan:
        plan.backward(gz.t, tokens.cuda(), lse.cuda(), entropy.cuda(), up(dlp), gd.t, dentropy=up(dh))
        torch.cuda.synchronize()
    gz.check_guards()
    gd.check_guards()
    want, off = reference_grad(z, tokens, lse, entropy, dlp, dh)
    u = ROUND[dtype]
    assert_near(gd.t, want, u * want.abs() + (1 + u) * off + TINY[dtype], "dlogits")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (5, 3), (7, 100), (300, 1003), (3, 50257), (2, 131072)])
def test_backward(rows, vocab, dtype):
    check_backward(rows, vocab, dtype)
    check_backward(rows, vocab, dtype, with_h=False)
    check_backward(rows, vocab, dtype, with_lp=False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("vocab,pitch,offset,d_offset", [(1000, 1008, 0, 0), (1001, 1001, 0, 0), (1000, 1003, 1, 2), (9001, 9008, 8, 5)])
def test_backward_pitches_and_offsets(vocab, pitch, offset, d_offset, dtype):
    check_backward(11, vocab, dtype, pitch=pitch, offset=offset, d_offset=d_offset)
    check_backward(11, vocab, dtype, pitch=pitch, offset=offset, same=True)


@pytest.mark.parametrize("dtype", DTYPES)
def test_backward_masks(dtype):
    z = normal((6, 4000), dtype, 25, 3.0)
    z[0] = -INF
    z[1, 10:] = -INF
    z[2] = torch.finfo(TORCH[dtype]).min
    z[4, ::3] = torch.finfo(TORCH[dtype]).min
    check_backward(6, 4000, dtype, z=z)


def test_backward_of_bad_tokens_and_nan_rows():
    z = normal((4, 300), "float32", 26).cuda()
    z[2, 5] = math.nan
    tokens = torch.tensor([0, 300, 1, 2]).cuda()
    lp, en, ls = (torch.empty(4, device="cuda") for _ in range(3))
    d, one = torch.empty_like(z), torch.ones(4, device="cuda")
    with TokenLogProbsPlan(4, 300, "float32") as plan:
        plan.forward(z, tokens, lp, entropy=en, lse=ls)
        plan.backward(z, tokens, ls, en, one, d, dentropy=one)
        nan = torch.isnan(d).all(-1).tolist()
        assert nan == [False, True, True, False] and torch.isfinite(d[[0, 3]]).all()


def test_gradient_matches_central_differences():
    # the loss' third derivative along v is below a few |w| |v|^3; with |v_j| ~ 1 and h = 2^-6 that is 1e-4 of the
    # scale, and float32 outputs over 2 h give 2^-24 * 64 * |loss| more
    rows, vocab, h = 5, 60, 2.0 ** -6
    z = normal((rows, vocab), "float32", 31, 2.0).cuda()
    tokens = tokens_of(rows, vocab, 32).cuda()
    w, x = normal((rows,), "float32", 33).cuda(), normal((rows,), "float32", 34).cuda()
    lp, en, ls = (torch.empty(rows, device="cuda") for _ in range(3))
    with TokenLogProbsPlan(rows, vocab, "float32") as plan:
        def loss(a):
            plan.forward(a, tokens, lp, entropy=en, lse=ls)
            return float((lp.double() * w.double() + en.double() * x.double()).sum())
        loss(z)
        d = torch.empty_like(z)
        plan.backward(z, tokens, ls, en, w, d, dentropy=x)
        for seed in range(6):
            v = normal((rows, vocab), "float32", 40 + seed).cuda()
            want = float((d.double() * v.double()).sum())
            got = (loss(z + h * v) - loss(z - h * v)) / (2 * h)
            assert abs(got - want) <= 4e-3 * float(w.norm() + x.norm()) * math.sqrt(rows)


def test_offsets_beyond_32_bits_streams_and_graph():
    rows, vocab, pitch = 3, 5000, 2 ** 30 + 64
    storage = torch.empty(2 * pitch + vocab, dtype=torch.float16, device="cuda")
    z = torch.as_strided(storage, (rows, vocab), (pitch, 1))
    z.copy_(normal((rows, vocab), "float16", 51, 3.0))
    tokens = tokens_of(rows, vocab, 52).cuda()
    far, near = token_log_probs(z, tokens, 5), token_log_probs(z.contiguous(), tokens, 5)
    assert all(torch.equal(a, b) for a, b in zip(far, near))
    dense, d = z.contiguous(), torch.empty(rows, vocab, dtype=torch.float16, device="cuda")
    lp, ls = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    one = torch.ones(rows, device="cuda")
    with TokenLogProbsPlan(rows, vocab, "float16") as plan:
        def step(stream=None):
            plan.forward(dense, tokens, lp, lse=ls, stream=stream)
            plan.backward(dense, tokens, ls, None, one, d, stream=stream)
        step()
        torch.cuda.synchronize()
        want = d.clone()
        plan.backward(z, tokens, ls, None, one, z)             # in place, beyond 32 bits
        assert torch.equal(z, want)
        s = torch.cuda.Stream()
        d.zero_()
        s.wait_stream(torch.cuda.current_stream())
        step(s)
        s.synchronize()
        assert torch.equal(d, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        d.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(d, want)


def test_refusals():
    z, tokens, lp = torch.zeros(4, 8, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(4, device="cuda")
    with TokenLogProbsPlan(4, 8, "float32", 2) as plan:
        for bad in (z.half(), z[:, :4], torch.zeros(4, 8)):
            with pytest.raises((TypeError, ValueError)):
                plan.forward(bad, tokens, lp)
        with pytest.raises(TypeError):
            plan.forward(z, tokens.int(), lp)
        with pytest.raises(ValueError):
            plan.forward(z, tokens, lp, top_index=torch.zeros(4, dtype=torch.int64, device="cuda"))
        with pytest.raises(OlcError) as e:
            plan.backward(z, None, lp, None, lp, z)
        assert e.value.name == "OLC_ERR_NULL"
        with pytest.raises(OlcError) as e:
            plan.backward(z, tokens, lp, None, lp, z, dentropy=lp)
        assert e.value.name == "OLC_ERR_NULL"
        lib, p = plan.lib, z.data_ptr()
        assert lib.olc_token_log_probs_forward(plan._h, p, 7, p, p, None, None, None, None, None) == 13
        assert lib.olc_token_log_probs_forward(plan._h, p, 8, p + 4, p, None, None, None, None, None) == 13
        assert lib.olc_token_log_probs_backward(plan._h, p, 8, p, p, None, p, None, p, 7, None) == 13
