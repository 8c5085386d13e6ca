"""What the tests of the layer plans share: unit roundoffs, tensors with a row
pitch or an odd start inside guarded storage, and a comparison by element."""

import torch

DTYPES = ["float32", "float16", "bfloat16"]
TORCH = {"float32": torch.float32, "float16": torch.float16, "bfloat16": torch.bfloat16}
#: largest relative error of one rounding to nearest, and the smallest absolute one
ROUND = {"float32": 2.0 ** -24, "float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}
TINY = {"float32": 2.0 ** -126, "float16": 2.0 ** -25, "bfloat16": 2.0 ** -126}
F32 = 2.0 ** -24
CANARY = 7.25


def normal(shape, dtype, seed, scale=1.0, shift=0.0):
    """The same values on every machine: drawn on the CPU."""
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale + shift).to(TORCH[dtype])


class Guarded:
    """A [rows, cols] CUDA matrix whose rows are `pitch` apart and whose start
    is `offset` elements into its storage; everything outside it holds a
    canary."""

    def __init__(self, rows, cols, dtype, pitch=None, offset=0, values=None):
        self.pitch, self.offset = pitch or cols, offset
        self.rows, self.cols = rows, cols
        span = max(0, (rows - 1) * self.pitch + cols) if rows else 0
        self.storage = torch.full((offset + span + 32,), CANARY, dtype=TORCH[dtype] if isinstance(dtype, str) else dtype,
                                  device="cuda")
        self.t = torch.as_strided(self.storage, (rows, cols), (self.pitch, 1), offset)
        if values is not None:
            self.t.copy_(values)

    def check_guards(self):
        inside = torch.zeros(self.storage.numel(), dtype=torch.bool, device="cuda")
        torch.as_strided(inside, (self.rows, self.cols), (self.pitch, 1), self.offset).fill_(True)
        assert (self.storage[~inside] == CANARY).all(), "written outside of the matrix"


def assert_near(got, want, tol, what):
    """|got - want| <= tol by element; NaN and infinities where and as `want` has them."""
    got, want = got.detach().double().cpu(), want.double().cpu()
    tol = tol.double().cpu() if isinstance(tol, torch.Tensor) else torch.full_like(want, tol)
    assert got.shape == want.shape, what
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "%s: NaN in other places" % what
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), "%s: infinities differ" % what
    fine = torch.isfinite(want)
    err = (got - want).abs()[fine]
    bad = ~(err <= tol[fine])
    assert not bad.any(), "%s: %d of %d off, worst %g of the tolerance" % (
        what, int(bad.sum()), bad.numel(), float((err / tol[fine])[bad].max()))
