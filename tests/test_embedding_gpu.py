"""Rows of a table by token id on the GPU, and the table's gradient, against the
definitions in 64 bits.

Tolerances.  Forward: one float32 product and one rounding to the element type.
Backward: a token's float32 sum over its n places, in whatever order, is off by at
most n 2^-24 times the sum of the magnitudes (n - 1 additions, the scale), plus an
addition and its product where the gradient is accumulated, and the one rounding to
the element type."""

import pytest
import torch

from gemm_matmulplan_broadcast_gb300 import EmbeddingPlan, OlcError, embedding
from layers_ref import DTYPES, F32, ROUND, TINY, TORCH, Guarded, assert_near, normal

pytestmark = pytest.mark.gpu

#: ids, tokens, columns: one of each; odd widths; places that cross many chunks; a sparse
#: vocabulary; more tokens than one sort block takes; several turns of the sort's loops
SIZES = [(1, 1, 1), (5, 7, 33), (700, 50, 64), (4096, 3, 96), (3000, 40000, 40), (33, 5000, 1000), (20000, 911, 16),
         (64, 300000, 8), (513, 2, 2049), (2500, 100, 4096), (900, 130, 1350), (70, 9, 2)]


def ids_of(n, vocab, seed, strange=True):
    g = torch.Generator().manual_seed(seed)
    ids = (vocab ** torch.rand(n, generator=g, dtype=torch.float64)).long().clamp(max=vocab) - 1     # low ids often
    if strange and n > 4:
        ids[torch.rand(n, generator=g) < 0.1] = -1
        ids[1], ids[2], ids[3] = -5, vocab, vocab + 2 ** 40
    return ids


def forward_want(table, ids, scale):
    y = torch.zeros(len(ids), table.shape[1], dtype=torch.float64)
    known = (ids >= 0) & (ids < table.shape[0])
    y[known] = table.double()[ids[known]] * scale
    y[ids >= table.shape[0]] = float("nan")
    return y


def backward_want(dy, ids, vocab, scale):
    known = (ids >= 0) & (ids < vocab)
    total, size, places = (torch.zeros(vocab, dy.shape[1], dtype=torch.float64) for _ in range(3))
    total.index_add_(0, ids[known], dy.double()[known] * scale)
    size.index_add_(0, ids[known], dy.double()[known].abs() * abs(scale))
    places.index_add_(0, ids[known], torch.ones(int(known.sum()), dy.shape[1], dtype=torch.float64))
    return total, size, places


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,cols", SIZES)
def test_forward(n, vocab, cols, dtype):
    table, ids, scale = normal((vocab, cols), dtype, 1), ids_of(n, vocab, 2), 1.0 if n % 2 else 12.5
    y = Guarded(n, cols, dtype)
    with EmbeddingPlan(n, vocab, cols, dtype, scale) as plan:
        plan.forward(table.cuda(), ids.cuda(), y.t)
        torch.cuda.synchronize()
    y.check_guards()
    want = forward_want(table, ids, scale)
    assert_near(y.t, want, want.abs() * (ROUND[dtype] + F32) + TINY[dtype], "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("n,vocab,cols", SIZES)
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward(n, vocab, cols, dtype, accumulate):
    dy, ids, scale = normal((n, cols), dtype, 3), ids_of(n, vocab, 4), 0.75
    old = normal((vocab, cols), dtype, 5)
    de = Guarded(vocab, cols, dtype, values=old)
    with EmbeddingPlan(n, vocab, cols, dtype, scale) as plan:
        gids = ids.cuda()
        plan.backward(dy.cuda(), gids, de.t, accumulate=accumulate)
        torch.cuda.synchronize()
        first = de.t.clone()
        de.t.copy_(old)
        plan.backward(dy.cuda(), gids, de.t, accumulate=accumulate)
        torch.cuda.synchronize()
    de.check_guards()
    assert torch.equal(first, de.t), "another result the second time"
    want, size, places = backward_want(dy, ids, vocab, scale)
    if accumulate:
        want, size = want + old.double(), size + old.double().abs()
        untouched = places[:, 0] == 0
        assert torch.equal(first.cpu()[untouched], old[untouched])
    tol = (places + 2) * F32 * size + want.abs() * ROUND[dtype] + TINY[dtype]
    assert_near(first, want, tol, "dtable")


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("ids", ["one", "none", "first", "last", "all"])
def test_backward_of_uneven_ids(ids, dtype):
    n, vocab, cols = 5000, 1234, 72
    t = {"one": torch.full((n,), 77), "none": torch.full((n,), -1), "first": torch.zeros(n, dtype=torch.long),
         "last": torch.full((n,), vocab - 1), "all": torch.arange(n) % vocab}[ids]
    dy = normal((n, cols), dtype, 6)
    de = Guarded(vocab, cols, dtype)
    with EmbeddingPlan(n, vocab, cols, dtype) as plan:
        plan.backward(dy.cuda(), t.cuda(), de.t)
    want, size, places = backward_want(dy, t, vocab, 1.0)
    assert_near(de.t, want, (places + 2) * F32 * size + want.abs() * ROUND[dtype] + TINY[dtype], "dtable")
    de.check_guards()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pitch,offset", [(72, 0), (67, 0), (64, 1), (80, 3), (72, 8), (66, 2), (74, 6)])
def test_pitches_and_offsets(pitch, offset, dtype):
    n, vocab, cols = 300, 90, 64
    table, dy, ids = normal((vocab, cols), dtype, 7), normal((n, cols), dtype, 8), ids_of(n, vocab, 9)
    e, y = Guarded(vocab, cols, dtype, pitch, offset, table), Guarded(n, cols, dtype, pitch, offset)
    gdy, de = Guarded(n, cols, dtype, pitch, offset, dy), Guarded(vocab, cols, dtype, pitch, offset)
    with EmbeddingPlan(n, vocab, cols, dtype, 2.0) as plan:
        plan.forward(e.t, ids.cuda(), y.t)
        plan.backward(gdy.t, ids.cuda(), de.t)
        torch.cuda.synchronize()
    for g in (e, y, gdy, de):
        g.check_guards()
    want = forward_want(table, ids, 2.0)
    assert_near(y.t, want, want.abs() * (ROUND[dtype] + F32) + TINY[dtype], "y")
    want, size, places = backward_want(dy, ids, vocab, 2.0)
    assert_near(de.t, want, (places + 2) * F32 * size + want.abs() * ROUND[dtype] + TINY[dtype], "dtable")


def test_gradient_against_differences():
    n, vocab, cols = 40, 9, 5
    table, ids, c = normal((vocab, cols), "float32", 1), ids_of(n, vocab, 2, strange=False), normal((n, cols), "float32", 3)
    with EmbeddingPlan(n, vocab, cols, "float32", 1.5) as plan:
        value = lambda t: float((plan.forward(t.cuda(), ids.cuda(), torch.empty(n, cols, device="cuda")).double().cpu()  # noqa: E731
                                 * c.double()).sum())
        de = plan.backward(c.cuda(), ids.cuda(), torch.empty(vocab, cols, device="cuda")).cpu()
        for v, j in [(0, 0), (3, 4), (8, 2)]:
            up, down = table.clone(), table.clone()
            up[v, j] += 0.5
            down[v, j] -= 0.5
            # linear: the difference is the slope, but for the roundings of the products
            assert abs(value(up) - value(down) - float(de[v, j])) < 1e-4


def test_sizes_of_nothing():
    for n, vocab, cols in [(0, 5, 8), (4, 0, 8), (4, 5, 0), (0, 0, 0)]:
        ids = torch.full((n,), 2, device="cuda")
        table = torch.ones(vocab, cols, device="cuda")
        with EmbeddingPlan(n, vocab, cols, "float32") as plan:
            y = plan.forward(table, ids, torch.full((n, cols), 3.0, device="cuda"))
            assert vocab > 0 or torch.isnan(y).all()
            de = plan.backward(torch.ones(n, cols, device="cuda"), ids, torch.full((vocab, cols), 3.0, device="cuda"))
            assert float(de.sum()) == (n * cols if vocab else 0)      # a table without rows has no sums
            plan.backward(torch.ones(n, cols, device="cuda"), ids, de, accumulate=True)
            assert float(de.sum()) == (2 * n * cols if vocab else 0)


def test_offsets_beyond_32_bits():
    vocab, cols, n = 600_000, 4096, 6
    table = torch.empty(vocab, cols, dtype=torch.bfloat16, device="cuda")
    ids = torch.tensor([vocab - 1, 0, 550_000, -1, vocab - 1, 524_288], device="cuda")
    rows = normal((n, cols), "bfloat16", 1).cuda()
    rows[4] = rows[0]
    table[ids[ids >= 0]] = rows[ids >= 0]
    with EmbeddingPlan(n, vocab, cols, "bfloat16") as plan:
        y = plan.forward(table, ids, torch.empty_like(rows))
        rows[3] = 0
        assert torch.equal(y, rows)
        table.fill_(1)
        plan.backward(rows, ids, table)
        assert torch.equal(table[ids[[1, 2, 5]]], rows[[1, 2, 5]]) and torch.equal(table[vocab - 1], rows[0] * 2)
        others = torch.ones(vocab, dtype=torch.bool, device="cuda")
        others[ids[ids >= 0]] = False
        assert int((table.view(torch.int16).amax(1)[others] != 0).sum()) == 0


def test_one_shot_and_graph_and_streams():
    table, ids = normal((100, 40), "float16", 1).cuda(), ids_of(60, 100, 2, strange=False).cuda()
    assert torch.equal(embedding(table, ids.view(6, 10), 2.0), (table[ids] * 2).view(6, 10, 40))
    dy = normal((60, 40), "float16", 3).cuda()
    with EmbeddingPlan(60, 100, 40, "float16") as plan:
        want = plan.backward(dy, ids, torch.empty_like(table)).clone()
        out, y = torch.empty_like(table), torch.empty_like(dy)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            plan.backward(dy, ids, out)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            plan.forward(table, ids, y)
            plan.backward(dy, ids, out)
        ids.copy_(ids.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, table[ids])
        assert torch.equal(out, plan.backward(dy, ids, torch.empty_like(table)))


def test_refusals():
    with EmbeddingPlan(4, 5, 8, "float16") as plan:
        t = lambda *s, of=torch.float16: torch.zeros(s, dtype=of, device="cuda")  # noqa: E731
        table, ids, y = t(5, 8), t(4, of=torch.int64), t(4, 8)
        for bad in [(t(5, 7), ids, y), (table, ids, t(3, 8)), (table, t(3, of=torch.int64), y), (table.cpu(), ids, y),
                    (table, ids.cpu(), y), (t(5, 8).t().contiguous().t(), ids, y)]:
            with pytest.raises(ValueError):
                plan.forward(*bad)
        for bad in [(table.float(), ids, y), (table, ids.int(), y), (table, ids, y.float())]:
            with pytest.raises(TypeError):
                plan.forward(*bad)
        lib, h = plan.lib, plan._h
        p = [x.data_ptr() for x in (table, ids, y)]
        assert lib.olc_embedding_forward(h, None, 8, p[1], p[2], 8, None) == 1
        assert lib.olc_embedding_forward(h, p[0], 7, p[1], p[2], 8, None) == 13
        assert lib.olc_embedding_forward(h, p[0] + 1, 8, p[1], p[2], 8, None) == 13
        assert lib.olc_embedding_forward(h, p[0], 8, p[1] + 4, p[2], 8, None) == 13
        assert lib.olc_embedding_backward(h, p[2], 8, None, p[0], 8, 0, None) == 1
        assert lib.olc_embedding_backward(h, p[2], 2 ** 61, p[1], p[0], 8, 0, None) == 13
        assert lib.olc_embedding_backward(None, p[2], 8, p[1], p[0], 8, 0, None) == 1
    with pytest.raises(OlcError):
        EmbeddingPlan(4, 2 ** 31, 8, "float16")
