"""Host-side checks of the embedding, residual norm and sampling plans (no GPU
needed, no kernel launched): creation arguments, refusals by code."""

import ctypes

import pytest

from gemm_matmulplan_broadcast_gb300 import EmbeddingPlan, OlcError, ResidualNormPlan, SamplePlan, binding

EMBED = [((-1, 5, 8), 1.0, "OLC_ERR_NEGATIVE_DIM"), ((4, -5, 8), 1.0, "OLC_ERR_NEGATIVE_DIM"),
         ((4, 5, -8), 1.0, "OLC_ERR_NEGATIVE_DIM"), ((2 ** 31, 5, 8), 1.0, "OLC_ERR_INVALID"),
         ((4, 2 ** 31, 8), 1.0, "OLC_ERR_INVALID"), ((4, 5, 2 ** 31), 1.0, "OLC_ERR_INVALID"),
         ((2 ** 31 - 70000, 5, 2 ** 31 - 70000), 1.0, "OLC_ERR_INVALID"), ((4, 5, 8), float("nan"), "OLC_ERR_INVALID"),
         ((4, 5, 8), float("inf"), "OLC_ERR_INVALID")]


@pytest.mark.parametrize("shape,scale,error", EMBED)
def test_embedding_plan_refuses(shape, scale, error):
    with pytest.raises(OlcError) as e:
        EmbeddingPlan(*shape, "float32", scale)
    assert e.value.name == error


RESIDUAL = [((-1, 8), {}, "OLC_ERR_NEGATIVE_DIM"), ((4, -8), {}, "OLC_ERR_NEGATIVE_DIM"), ((4, 0), {}, "OLC_ERR_INVALID"),
            ((4, 2 ** 31), {}, "OLC_ERR_INVALID"), ((4, 8), {"eps": -1.0}, "OLC_ERR_INVALID"),
            ((4, 8), {"eps": float("nan")}, "OLC_ERR_INVALID"), ((4, 8), {"scale": float("inf")}, "OLC_ERR_INVALID"),
            ((2 ** 60, 2 ** 10), {}, "OLC_ERR_INVALID")]


@pytest.mark.parametrize("shape,kw,error", RESIDUAL)
def test_residual_norm_plan_refuses(shape, kw, error):
    with pytest.raises(OlcError) as e:
        ResidualNormPlan(*shape, "float32", **kw)
    assert e.value.name == error


SAMPLE = [((-1, 8), "OLC_ERR_NEGATIVE_DIM"), ((4, -8), "OLC_ERR_NEGATIVE_DIM"), ((4, 0), "OLC_ERR_INVALID"),
          ((4, 2 ** 20 + 1), "OLC_ERR_INVALID"), ((2 ** 27, 8), "OLC_ERR_INVALID")]


@pytest.mark.parametrize("shape,error", SAMPLE)
def test_sample_plan_refuses(shape, error):
    with pytest.raises(OlcError) as e:
        SamplePlan(*shape, "float32")
    assert e.value.name == error


def test_types_and_names():
    for make in (lambda t: EmbeddingPlan(4, 5, 8, t), lambda t: ResidualNormPlan(4, 8, t), lambda t: SamplePlan(4, 8, t)):
        for t in ("float32", "float16", "bfloat16"):
            make(t).close()
        for t in ("float64", "float8_e4m3fn", "int8"):
            with pytest.raises(ValueError):
                make(t)
    with pytest.raises(ValueError):
        ResidualNormPlan(4, 8, "float32", norm="batch")
    lib, h = binding.load(), ctypes.c_void_p()
    for code in (11, 17, 0, -1):
        assert lib.olc_embedding_plan_create(4, 5, 8, 1.0, code, ctypes.byref(h)) == 6 and not h.value
        assert lib.olc_residual_norm_plan_create(4, 8, 1e-5, 1.0, 0, 0, code, ctypes.byref(h)) == 6 and not h.value
        assert lib.olc_sample_plan_create(4, 8, code, ctypes.byref(h)) == 6 and not h.value
    assert lib.olc_residual_norm_plan_create(4, 8, 1e-5, 1.0, 2, 0, 1, ctypes.byref(h)) == 13
    assert lib.olc_embedding_plan_create(4, 5, 8, 1.0, 1, None) == 1
    assert lib.olc_residual_norm_plan_create(4, 8, 1e-5, 1.0, 0, 0, 1, None) == 1
    assert lib.olc_sample_plan_create(4, 8, 1, None) == 1
    for destroy in (lib.olc_embedding_plan_destroy, lib.olc_residual_norm_plan_destroy, lib.olc_sample_plan_destroy):
        destroy(None)


def test_calls_without_work_need_no_pointers():
    n = None
    with EmbeddingPlan(0, 5, 8, "float16") as p:
        assert p.lib.olc_embedding_forward(p._h, n, 8, n, n, 8, n) == 0
        assert p.lib.olc_embedding_backward(p._h, n, 8, n, n, 8, 1, n) == 0
        assert p.lib.olc_embedding_backward(p._h, n, 8, n, n, 8, 0, n) == 1          # zeros have to go somewhere
    with ResidualNormPlan(0, 8, "float16", after=True) as p:
        assert p.lib.olc_residual_norm_forward(p._h, n, 8, n, 8, n, 0, n, n, n, n, n, 8, n, 8, n, n) == 0
        assert p.lib.olc_residual_norm_backward(p._h, n, 8, n, 8, n, 8, n, 8, n, n, 0, n, n, n, n, 8, n, 8, n, 0, n, n, n,
                                                n, n) == 0
    with SamplePlan(0, 8, "float16") as p:
        assert p.lib.olc_sample_forward(p._h, n, 8, n, n, n, n, n, n, n, n) == 0


def test_refusals_before_any_device_work():
    n, p8 = None, 4096                                     # an address that is never read
    with ResidualNormPlan(4, 8, "float16", after=True) as p:
        call = lambda dy, dz, f, y, stats, gate, dx, dgate, dgamma: p.lib.olc_residual_norm_backward(  # noqa: E731
            p._h, dy, 8, dz, 8, f, 8, y, 8, stats, gate, 0, n, n, n, dx, 8, n, 8, dgate, 0, dgamma, n, n, n, n)
        assert call(n, n, p8, p8, p8, n, p8, n, n) == 1            # neither gradient
        assert call(p8, n, n, p8, p8, n, p8, n, n) == 1            # no F with the norm of F
        assert call(p8, p8, p8, n, p8, n, p8, n, n) == 1           # no Y with dZ
        assert call(p8, p8, p8, p8, n, n, p8, n, n) == 1           # no stats
        assert call(p8, n, p8, p8, p8, n, p8, n, p8) == 1          # dgamma without dZ
        assert call(p8, p8, p8, p8, p8, n, p8, p8, n) == 1         # dgate without a gate
        assert call(p8 + 1, p8, p8, p8, p8, n, p8, n, n) == 13
        assert call(p8, p8, p8, p8, p8 + 2, n, p8, n, n) == 13
        assert call(p8, p8, p8, p8, p8, p8 + 1, p8, n, n) == 13
    with ResidualNormPlan(4, 8, "float16") as p:
        assert p.lib.olc_residual_norm_backward(p._h, p8, 8, n, 8, n, 8, n, 8, n, n, 0, n, n, n, n, 8, n, 8, n, 0, n, n, p8,
                                                n, n) == 13
    with SamplePlan(4, 8, "float32") as p:
        for bad in range(8):
            a = [p8, p8, p8, p8, p8, p8, p8, p8]
            a[bad] += 2 if bad != 6 else 4
            z, u, t, k, tp, mp, tok, lp = a
            assert p.lib.olc_sample_forward(p._h, z, 8, u, t, k, tp, mp, tok, lp, n) == 13, bad
