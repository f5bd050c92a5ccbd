"""Angles p * f, p an integer and f a 32-bit float, in exact arithmetic: less whole turns before anything is rounded."""
import math
from fractions import Fraction

BITS = 400  # of pi; p * f has at most 159 before the point


def _pi():
    """pi by Machin's formula, 16 (arc cot 5) - 4 (arc cot 239), in integers."""
    one = 1 << (BITS + 20)

    def arc_cot(k):
        total = term = one // k
        n, sign = 1, -1
        while term:
            term //= k * k
            n += 2
            total += sign * (term // n)
            sign = -sign
        return total

    return Fraction(4 * (4 * arc_cot(5) - arc_cot(239)), one)


PI = _pi()


def cos_sin(p: int, f: float):
    """(cos, sin) of p * f radians, off by a few 2^-53."""
    angle = Fraction(p) * Fraction(f)
    angle -= round(angle / (2 * PI)) * 2 * PI
    angle = angle.numerator / angle.denominator  # rounded once
    return math.cos(angle), math.sin(angle)
