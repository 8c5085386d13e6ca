"""Layer norm of rows of equal values: what is left after the mean is nothing,
whatever the value and the width, in every kernel of the forward pass."""

import pytest
import torch

from layers_ref import DTYPES, F32, TORCH, Guarded, normal
from test_layer_norm_gpu import EPS, run_forward

pytestmark = pytest.mark.gpu

#: rows and widths that reach the kernel of short rows, a warp a row, several warps a row (16-byte packs and single
#: elements), and rows longer than a block's registers
SHAPES = [(5000, 24), (5000, 104), (9, 190), (9, 41), (700, 1000), (9, 1000), (9, 4097), (700, 4104), (9, 20000), (3, 40000),
          (3, 70001)]
VALUES = {"float32": [0.1, 3.0, 100.0, 1000.0, 1000.1, -77777.7], "float16": [0.1, 3.0, 1000.0, -60000.0],
          "bfloat16": [0.1, 3.0, 100.0, 1000.0, 77777.7]}
#: what the squares of the first mean's error, 256 2^-24 of the value, leave when they are taken out again: 256 2^-24 of
#: themselves, as a distance
LEFT = (256 * F32) ** 1.5


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_equal_values_leave_the_bias(rows, cols, dtype):
    beta = normal((cols,), dtype, 2)
    for value in VALUES[dtype]:
        x = torch.full((rows, cols), value).to(TORCH[dtype])
        for offset in (0, 1):
            y, mean, rstd = run_forward(x, normal((cols,), dtype, 1, 0.3, 1.0), beta, dtype, offset=offset)
            assert torch.equal(mean.cpu(), x[:, 0].float()), (value, offset)
            assert torch.equal(y.cpu(), beta.expand(rows, cols)), (value, offset)
            # the variance is nothing but the square of the mean's rounding, taken out again
            assert float((rstd * EPS ** 0.5 - 1).abs().max()) <= 4 * F32 + (LEFT * value) ** 2 / EPS, (value, offset)


@pytest.mark.parametrize("cols", [64, 190, 1000, 4097, 40000])
def test_equal_values_without_eps_divide_by_zero(cols):
    # sums that are exact: a variance of zero, so NaN (0 times infinity) in every column
    for value in (3.0, 100.0, 1000.0):
        x = torch.full((3, cols), value)
        y, mean, rstd = run_forward(x, None, None, "float32", eps=0.0)
        assert torch.isnan(y).all() and torch.isinf(rstd).all() and (mean == value).all(), value


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_the_mean_is_its_nearest_value(rows, cols, dtype):
    """Rows far from zero: the mean that the second pass corrects is off by
    one rounding of itself and by roundings of the distances from it."""
    x = normal((rows, cols), dtype, 5, 1.0, 300.0)
    y, mean, rstd = run_forward(x, None, None, dtype)
    want = x.double().mean(-1)
    spread = (x.double() - want[:, None]).abs().mean(-1)
    assert ((mean.double().cpu() - want).abs() <= F32 * want.abs() * 1.01 + 256 * F32 * spread).all()
