"""The plain forms of the layer operators against their own definitions on the CPU:
gradients against differences, codes against their properties."""
import numpy as np
import pytest

from oracle import layers


@pytest.mark.parametrize("name", layers.ACTS)
def test_slope_is_the_difference_quotient(name):
    """Central difference with h = 2^-17: truncation h^2/6 |f'''| (|f'''| <= 4) below 4e-11,
    rounding 2^-52 |f| / h below 3e-10 for |z| <= 8."""
    z = np.linspace(-8, 8, 1001) + 1e-3   # no point within h of relu's corner
    h = 2.0 ** -17
    diff = (layers.act(z + h, name) - layers.act(z - h, name)) / (2 * h)
    np.testing.assert_allclose(layers.slope(z, name), diff, rtol=0, atol=1e-9)


def test_layernorm_backward_is_the_difference_quotient():
    """The same for sum(dy * layernorm(x)): third derivatives of order 10 at these values, so
    h = 2^-16 leaves 1e-9 of truncation and 1e-10 of rounding."""
    rng = np.random.default_rng(1)
    x, dy = rng.standard_normal((3, 7)), rng.standard_normal((3, 7))
    gamma, beta = rng.standard_normal(7), rng.standard_normal(7)
    f = lambda x, g, b: float((dy * layers.layernorm(x, g, b)[0]).sum())
    _, mean, rstd = layers.layernorm(x, gamma, beta)
    dx, dgamma, dbeta = layers.layernorm_backward(dy, x, gamma, mean, rstd)
    h = 2.0 ** -16
    for i in range(3):
        for j in range(7):
            e = np.zeros_like(x)
            e[i, j] = h
            assert abs((f(x + e, gamma, beta) - f(x - e, gamma, beta)) / (2 * h)
                       - dx[i, j]) < 1e-7
    for j in range(7):
        e = np.zeros(7)
        e[j] = h
        assert abs((f(x, gamma + e, beta) - f(x, gamma - e, beta)) / (2 * h) - dgamma[j]) < 1e-8
        assert abs((f(x, gamma, beta + e) - f(x, gamma, beta - e)) / (2 * h) - dbeta[j]) < 1e-8


def test_codes():
    y = np.array([[1.0, -2.0, 0.5, 0.0], [0, 0, 0, 0], [1, np.inf, 0, 0], [1, np.nan, 0, 0],
                  [1e300, 1, 0, 0], [1e-60, 0, 0, 0]])
    quot, scale = layers.int8_codes(y)
    assert scale[0] == np.float32(2 / 127) and np.rint(quot[0]).tolist() == [64, -127, 32, 0]
    assert scale[1] == 0 and scale[5] == 0 and not quot[1].any() and not quot[5].any()
    assert np.isnan(scale[2:5]).all() and not quot[2:5].any()


def test_int8_linear_sums_are_exact():
    x = np.full((2, 131071), -128, dtype=np.int8)
    assert layers.int8_sums(x, x)[0, 1] == 131071 * 16384
