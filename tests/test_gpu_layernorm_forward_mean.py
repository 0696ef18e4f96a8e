"""Rows whose sum is exact have an exact mean: the LayerNorm forward of a constant row
is the bias, whatever the width."""
import numpy as np
import pytest

import linear_layer_gemms_gb300 as mm
from test_gpu_layernorm_forward import call, host, lib  # noqa: F401

pytestmark = pytest.mark.gpu


# a width of every kernel variant, none whose reciprocal is near a number of fp32
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("C", [776, 1008, 2016, 4032, 8160, 16_320, 32_640, 65_520, 95_432])
def test_constant_rows_give_the_bias(C, dtype):
    """Multiples of 1/8 up to 2^24 / C, so that every partial sum is exact in fp32 (and
    up to 255 / 8 in bf16): the mean is the constant, the differences are zero."""
    g = np.random.default_rng(C)
    top = min((1 << 24) // C, 255 if dtype == "bf16" else 4095)
    k = np.unique(g.integers(1, top + 1, 200))
    x = np.repeat(k[:, None] / 8.0, C, 1)
    x[::2] *= -1
    w, b = np.full(C, 1.5), g.integers(-32, 33, C) / 8.0
    out, mean, rstd = call(x, w, b, 1e-5, dtype)
    np.testing.assert_array_equal(host(mean), x[:, 0])
    np.testing.assert_array_equal(host(out), np.broadcast_to(b, x.shape))
    want = 1 / np.sqrt(float(np.float32(1e-5)))  # of eps as the call takes it: a root and a quotient, half a step each
    assert np.all(np.abs(host(rstd) - want) <= 2.001 * 2.0 ** -24 * want)


@pytest.mark.parametrize("C", [776, 8160, 95_432])
def test_the_mean_of_an_infinite_sum_is_infinite(C):
    x = np.ones((4, C))
    x[0, 5], x[1, C - 1], x[2, 7] = np.inf, -np.inf, np.nan
    _, mean, _ = call(x, np.ones(C), np.zeros(C), 1e-5, "f32")
    np.testing.assert_array_equal(host(mean), [np.inf, -np.inf, np.nan, 1.0])
