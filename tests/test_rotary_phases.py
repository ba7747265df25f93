"""Frequencies as 64-bit fractions of a turn against integer arithmetic (no GPU)."""
from fractions import Fraction

import numpy as np
import pytest

from test_ops_abi import kda  # noqa: F401  (the fixture)

PI = Fraction(314159265358979323846264338327950288419716939937510582097494459, 10 ** 62)      # to 62 digits, 2^-205


@pytest.mark.parametrize("theta", [10000.0, 500000.0, 1e6])
@pytest.mark.parametrize("rot", [16, 64, 128, 256])
def test_every_bit_of_the_usual_frequencies(theta, rot, kda):  # noqa: F811
    """The word is the fraction to one step of 2^-64, half of it from the last rounding: times 2^31 positions the angle is off by 2^-33 of a
    turn, 7.3e-10, at most."""
    _check(theta ** (-np.arange(0, rot, 2) / rot), kda)


def test_every_bit_of_other_frequencies(kda):  # noqa: F811
    rng = np.random.RandomState(0)
    f = np.concatenate([rng.randn(200) * 10.0 ** rng.uniform(-25, 9, 200), [np.pi, 2 * np.pi, -np.pi, 1e-300, -1e-300, 5e-324, -1e-25, 0.0, -0.0, 1.0, -1.0]])
    _check(f, kda)


def test_any_finite_frequency(kda):  # noqa: F811
    """From 2^42 on the fraction's lowest bits are those of 107 bits of the quotient."""
    f = np.array([1e12, -3.7e14, 1e20, -1e22])
    _check(f, kda, relative=Fraction(1, 2 ** 105))
    assert kda.kda_rotary_phases([1e300, -1.7e308]).shape == (2,)


def _check(f, kda, relative=0):  # noqa: F811
    words = kda.kda_rotary_phases(f).view(np.uint64)
    for x, word in zip(f.tolist(), words.tolist()):
        turns = Fraction(x) / (2 * PI)
        gap = (Fraction(word) - turns * 2 ** 64) % 2 ** 64
        assert min(gap, 2 ** 64 - gap) <= 1 + abs(turns) * relative * 2 ** 64, x
