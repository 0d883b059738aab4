"""The plain forms of the feed-forward operators against their own definitions on the CPU."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import feedforward as ff
from oracle import layers


def nearest(v: float) -> int:
    """The code of |v|'s nearest value by exact distances, ties to the even code."""
    d = [abs(Fraction(abs(v)) - Fraction(float(g))) for g in ff.GRID]
    best = min(d)
    codes = [c for c in range(8) if d[c] == best]
    return codes[0] if len(codes) == 1 else next(c for c in codes if c % 2 == 0)


def test_codes_are_the_nearest_values():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((6, 300)) * np.exp(rng.standard_normal((6, 1)))
    x[1, :64] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], 8)   # every midpoint
    x[1, 32:64] *= -1
    x[2, 64:96] = 0
    x[3] *= 1e-300
    codes, scales = ff.mx_quant(x)
    assert codes.shape == (6, 512) and scales.shape == (6, 16) and not codes[:, 300:].any()
    for i in range(6):
        for b in range(9):
            block = x[i, 32 * b:32 * b + 32]
            e = int(scales[i, b]) - 127
            amax = np.abs(block).max()
            if amax > 0:
                exact = Fraction(amax)
                p = Fraction(2) ** (e + 2)
                assert p <= exact < 2 * p or (e == -127 and exact < 2 * p)
            else:
                assert e == -127
            for u, v in enumerate(block):
                c = int(codes[i, 32 * b + u])
                assert c & 7 == nearest(float(Fraction(v) / Fraction(2) ** e))
                assert (c >> 3) == int(np.signbit(v))


def test_blocks_without_a_scale():
    x = np.ones((4, 96))
    x[0, 3], x[1, 40], x[2, 70], x[3, 95] = np.inf, np.nan, 2.0 ** 130, -2.0 ** 129
    codes, scales = ff.mx_quant(x)
    assert [list(np.flatnonzero(s == 255)) for s in scales] == [[0], [1], [2], []]
    assert not codes[0, :32].any() and codes[3, 95] == 8 + 6 and scales[3, 2] == 254
    assert np.isnan(ff.mx_values(codes, scales)[0, :32]).all()


def test_values_invert_codes():
    codes = np.tile(np.arange(16, dtype=np.uint8), 32)[None]
    scales = np.arange(120, 136, dtype=np.uint8)[None]
    v = ff.mx_values(codes, scales)
    c2, s2 = ff.mx_quant(v)   # every block holds a 6: the same exponent
    np.testing.assert_array_equal(s2, scales)
    np.testing.assert_array_equal(c2, codes)
    np.testing.assert_array_equal(ff.mx_unpack(ff.mx_pack(codes)), codes)


@pytest.mark.parametrize("name", layers.ACTS)
def test_gate_grad_is_the_difference_quotient(name):
    """Central difference with h = 2^-17 of products of act (third derivative at most 4) with
    a linear factor of at most 4: h^2 / 6 * 16 + 2^-52 * 50 / h below 4e-9."""
    rng = np.random.default_rng(3)
    z, dc = rng.standard_normal((4, 6)), rng.standard_normal((4, 3))
    f = lambda z: float((dc * ff.gate(z, name)).sum())
    g = ff.gate_grad(dc, z, name)
    h = 2.0 ** -17
    for at in np.ndindex(z.shape):
        e = np.zeros_like(z)
        e[at] = h
        assert abs((f(z + e) - f(z - e)) / (2 * h) - g[at]) < 4e-9


def test_clip():
    norm, out = ff.clip([np.array([3.0]), np.array([[4.0, 0.0]])], 1.0)
    assert norm == 5.0 and out[0][0] == 0.6000000000000001 and out[1][0, 0] == 0.8
    norm, out = ff.clip([np.array([3e200, 4e200])], 10.0)
    np.testing.assert_allclose(norm, 5e200, rtol=1e-15)
    np.testing.assert_allclose(out[0], [6.0, 8.0], rtol=1e-15)
    norm, out = ff.clip([np.array([3e-200, 4e-200])], 1.0)
    np.testing.assert_allclose(norm, 5e-200, rtol=1e-15)
    np.testing.assert_array_equal(out[0], [3e-200, 4e-200])
    assert ff.clip([np.array([1.0, np.inf])], 1.0)[0] == np.inf
    assert np.isnan(ff.clip([np.array([1.0, np.nan])], 1.0)[0])
