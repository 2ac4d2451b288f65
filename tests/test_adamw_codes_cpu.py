"""How far the 8-bit rounding of r = sqrt(v) can lag behind its gradients, from
the coding alone."""
import math

import numpy as np
import pytest

import adamw_reference as ref


def frozen_factor(b2):
    """Most by which a stored r can stay too small for a constant gradient.

    With d = 2^-9 scales, r at code k < 8 stands for k*d (below 2^-6 scales the
    codes are d apart) and a step makes it x = sqrt(b2 k^2 + (1-b2) G^2) d for
    a gradient G d. The noise carries x to at most the next eighth of its
    octave, and that goes to the nearest whole number, ties to even. So it
    stays at k for certain while x is at most the eighth below the first one
    that rounds up: 1.375 for k = 1 (eighths of 1 to 2: 1.5 rounds to 2),
    2.5 for 2 (steps of 1/4: 2.5 rounds to 2, 2.75 to 3), 3.25 for 3, 4.5 for 4
    (steps of 1/2: 4.5 to 4), 5 for 5 (5.5 to 6), 6.5 for 6, 7 for 7. G / k is
    largest for k = 1."""
    last = {1: 1.375, 2: 2.5, 3: 3.25, 4: 4.5, 5: 5.0, 6: 6.5, 7: 7.0}
    return max(math.sqrt((x * x - b2 * k * k) / (1.0 - b2)) / k for k, x in last.items())


def _code(k, x, noise):
    """The code that k's successor x is stored as, in units of 2^-9 scales."""
    return ref.code_value(np.ldexp(x, -9), noise, np.zeros(x.shape, int), True) * 512.0


@pytest.mark.parametrize("b2,stated", [(0.95, 4.4), (0.99, 9.6), (0.999, 29.9)])
def test_the_stated_factor_is_where_codes_stop_moving(b2, stated):
    """Over all the noise: at each code below 8 the largest gradient under
    which no noise moves it is the derived one, and none exceeds the factor."""
    assert frozen_factor(b2) <= stated <= 1.02 * frozen_factor(b2)
    noise = np.arange(65536.0)
    for k in range(1, 8):
        low, high = k * 1.0, 1000.0 * k         # G that leaves k where it is, G that moves it
        for _ in range(60):
            g = 0.5 * (low + high)
            x = np.full(65536, math.sqrt(b2 * k * k + (1.0 - b2) * g * g))
            stays = (_code(k, x, noise) == k).all()
            low, high = (g, high) if stays else (low, g)
        assert low / k <= frozen_factor(b2) * (1 + 1e-4), (k, low / k)
        if k == 1:
            assert low / k >= frozen_factor(b2) * (1 - 1e-4)


def test_three_mantissa_bits_never_stop_moving():
    """From 2^-6 scales on, a gradient above r moves it up for some noise, and
    one below moves it down, however close: to the sixteen bits of the noise."""
    noise = np.arange(65536.0)
    for k in (9.0, 13.0, 16.0, 100.0):
        for up in (True, False):
            got = _code(k, np.full(65536, k * (1.001 if up else 0.999)), noise)
            assert (got > k).any() if up else (got < k).any()
            assert abs(got.mean() / (k * (1.001 if up else 0.999)) - 1) < 2.0 ** -16
