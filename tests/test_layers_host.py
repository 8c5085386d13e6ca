"""Host-side checks of the layer plans (no GPU needed, no kernel launched):
creation arguments, refusals by code."""

import ctypes

import pytest

from gemm_matmulplan_broadcast_gb300 import GatedPlan, LayerNormPlan, OlcError, TokenLogProbsPlan, binding

CREATE_NORM = [
    ((4, 0), "float32", 1e-5, "OLC_ERR_INVALID"),          # the mean of nothing
    ((4, 2 ** 31), "float32", 1e-5, "OLC_ERR_INVALID"),
    ((-1, 8), "float32", 1e-5, "OLC_ERR_NEGATIVE_DIM"),
    ((4, -8), "float32", 1e-5, "OLC_ERR_NEGATIVE_DIM"),
    ((4, 8), "float32", -1.0, "OLC_ERR_INVALID"),
    ((4, 8), "float32", float("nan"), "OLC_ERR_INVALID"),
    ((4, 8), "float32", float("inf"), "OLC_ERR_INVALID"),
    ((2 ** 60, 2 ** 10), "float32", 1e-5, "OLC_ERR_INVALID"),
]


@pytest.mark.parametrize("shape,dtype,eps,error", CREATE_NORM)
def test_layer_norm_plan_refuses(shape, dtype, eps, error):
    with pytest.raises(OlcError) as e:
        LayerNormPlan(*shape, dtype, eps)
    assert e.value.name == error


def test_layer_plans_take_three_types():
    for dtype in ("float32", "float16", "bfloat16"):
        LayerNormPlan(0, 1, dtype).close()
    for dtype in ("float64", "float8_e4m3fn", "int8"):
        with pytest.raises(ValueError):
            LayerNormPlan(4, 8, dtype)
    lib, h = binding.load(), ctypes.c_void_p()
    for code in (11, 17, 0, -1):
        assert lib.olc_layer_norm_plan_create(4, 8, 1e-5, code, ctypes.byref(h)) == 6 and not h.value
    assert lib.olc_layer_norm_plan_create(4, 8, 1e-5, 1, None) == 1
    lib.olc_layer_norm_plan_destroy(None)


def test_layer_norm_plan_rows_of_zero_need_no_pointers():
    with LayerNormPlan(0, 8, "bfloat16") as plan:
        assert plan.lib.olc_layer_norm_forward(plan._h, None, 8, None, None, None, 8, None, None, None) == 0
        assert plan.lib.olc_layer_norm_backward(plan._h, None, 8, None, 8, None, None, None, None, 8, None, None,
                                                None) == 0


CREATE_SCORE = [
    (4, 0, 0, "OLC_ERR_INVALID"),
    (4, 2 ** 31, 0, "OLC_ERR_INVALID"),
    (2 ** 27, 8, 0, "OLC_ERR_INVALID"),
    (4, 8, 9, "OLC_ERR_INVALID"),               # more alternatives than tokens
    (4, 100, 33, "OLC_ERR_INVALID"),
    (4, 100, -1, "OLC_ERR_INVALID"),
    (-4, 100, 0, "OLC_ERR_NEGATIVE_DIM"),
    (4, -100, 0, "OLC_ERR_NEGATIVE_DIM"),
]


@pytest.mark.parametrize("rows,vocab,top,error", CREATE_SCORE)
def test_token_log_probs_plan_refuses(rows, vocab, top, error):
    with pytest.raises(OlcError) as e:
        TokenLogProbsPlan(rows, vocab, "float16", top)
    assert e.value.name == error


def test_token_log_probs_plan_of_no_rows_needs_no_pointers():
    lib, h = binding.load(), ctypes.c_void_p()
    for code in (11, 17, 0):
        assert lib.olc_token_log_probs_plan_create(4, 8, 0, code, ctypes.byref(h)) == 6 and not h.value
    assert lib.olc_token_log_probs_plan_create(4, 8, 0, 1, None) == 1
    lib.olc_token_log_probs_plan_destroy(None)
    with TokenLogProbsPlan(0, 8, "bfloat16", 8) as plan:
        assert lib.olc_token_log_probs_forward(plan._h, None, 8, None, None, None, None, None, None, None) == 0
        assert lib.olc_token_log_probs_backward(plan._h, None, 8, None, None, None, None, None, None, 8, None) == 0


CREATE_GATED = [
    ((-1, 8, 8), "OLC_ERR_NEGATIVE_DIM"),
    ((4, -8, 8), "OLC_ERR_NEGATIVE_DIM"),
    ((4, 8, -8), "OLC_ERR_NEGATIVE_DIM"),
    ((2 ** 31, 8, 8), "OLC_ERR_INVALID"),
    ((4, 2 ** 31, 8), "OLC_ERR_INVALID"),
    ((4, 8, 2 ** 31), "OLC_ERR_INVALID"),
]


@pytest.mark.parametrize("sizes,error", CREATE_GATED)
def test_gated_plan_refuses(sizes, error):
    for dtype in ("float32", "bfloat16"):
        with pytest.raises(OlcError) as e:
            GatedPlan(*sizes, dtype)
        assert e.value.name == error


def test_gated_plan_arguments_and_empty_calls():
    lib, h = binding.load(), ctypes.c_void_p()
    with pytest.raises(ValueError):
        GatedPlan(4, 8, 8, "float32", act="tanh")
    for act in (-1, 4):
        assert lib.olc_gated_plan_create(4, 8, 8, act, 0, 1, ctypes.byref(h)) == 13 and not h.value
    for code in (11, 17, 0):
        assert lib.olc_gated_plan_create(4, 8, 8, 0, 0, code, ctypes.byref(h)) == 6 and not h.value
    assert lib.olc_gated_plan_create(4, 8, 8, 0, 0, 1, None) == 1
    lib.olc_gated_plan_destroy(None)
    no = [None] * 8
    for sizes in ((0, 8, 8), (4, 8, 0)):
        with GatedPlan(*sizes, "float16") as plan:
            assert lib.olc_gated_forward(plan._h, *no[:7]) == 0
    with GatedPlan(0, 0, 8, "float16") as plan:
        assert lib.olc_gated_backward(plan._h, *no, None, None) == 0
    with GatedPlan(4, 8, 8, "float16") as plan:
        assert lib.olc_gated_forward(plan._h, *no[:7]) == 1
        assert lib.olc_gated_backward(plan._h, *no, 16, None) == 1       # one weight's gradient alone
