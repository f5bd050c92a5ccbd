"""The exact angles against the C library's cosine and sine of the same products, where 64 bits hold them."""
import math
import random
from fractions import Fraction

import pytest

from tests import angle_ref


@pytest.mark.parametrize("low,high", [(-40, 0), (0, 20), (20, 100)])
def test_exact_angles(low, high):
    rng = random.Random(high)
    for _ in range(200):
        p = rng.randint(-2 ** 31, 2 ** 31 - 1)
        f = math.ldexp(rng.randint(2 ** 20, 2 ** 21), rng.randint(low, high) - 21)  # 31 + 21 bits
        assert Fraction(p * f) == Fraction(p) * Fraction(f)
        for got, want in zip(angle_ref.cos_sin(p, f), (math.cos(p * f), math.sin(p * f))):
            assert abs(got - want) <= 4 * 2.0 ** -53


def test_turns_of_pi():
    assert abs(float(angle_ref.PI) - math.pi) == 0
    assert angle_ref.cos_sin(0, 3e38) == (1.0, 0.0)
    # the float next to pi: sin of it is the distance, known to be -8.74e-8
    c, s = angle_ref.cos_sin(1, 3.1415927410125732)
    assert abs(c + 1) < 1e-14
    assert abs(s - (math.pi - 3.1415927410125732)) < 1e-15
