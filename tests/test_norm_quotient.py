"""The quotient that the blockwise norm rounds to 8 bits: one correction step of q0 = RN(y * RN(1/s)) for binary32 y and s.

With t = y / s, q0 is within 2^-23 of t, relative.  The residual and RN(1/s) carry 2^-24 each, so that the value that
the step rounds is within 2^-23 * 2^-23 of t, relative: 2^-21 half-ulps, as t is below 2^25 of them.  It rounds to
another binary32 than t only if a midpoint X of two neighbours lies between, and the two then give different 8-bit codes
only if one of them is a value m between two codes (at most 5 significant bits: 4 of e4m3 and one more; fewer for e5m2
and for subnormals), so X = m * 2^20 +- 1 half-ulps with m in 16 .. 32.  For Y and S, the significands as integers of 24
bits, and c = 24 or 25: |t - X| <= 2^-21 means |Y * 2^c - X * S| < 8.  X is odd, so each remainder gives one S: all of
them are tried here, up to a remainder of 64, in exact arithmetic.  Powers of two and signs only scale the sequence."""
from fractions import Fraction


def rn(x):
    """The nearest number of 24 significant bits, ties to even."""
    if x == 0:
        return x
    sign, x = (1, x) if x > 0 else (-1, -x)
    e = x.numerator.bit_length() - x.denominator.bit_length()
    if Fraction(2) ** e > x:
        e -= 1
    unit = Fraction(2) ** (e - 23)
    k, rest = divmod(x, unit)
    if 2 * rest > unit or (2 * rest == unit and k % 2):
        k += 1
    return sign * k * unit


def near_a_boundary(most):
    for m in range(16, 33):
        for x in (m * 2 ** 20 - 1, m * 2 ** 20 + 1):
            if not 2 ** 24 <= x < 2 ** 25:
                continue
            for c in (24, 25):
                inverse = pow(x, -1, 2 ** c)
                for e in range(-most, most + 1):
                    s = e * inverse % 2 ** c
                    y = (x * s - e) >> c
                    if 2 ** 23 <= s < 2 ** 24 and 2 ** 23 <= y < 2 ** 24:
                        assert y * 2 ** c == x * s - e
                        yield y, s


def test_one_step_is_enough_for_the_codes():
    tried = without = 0
    for y, s in near_a_boundary(64):
        y, s = Fraction(y), Fraction(s)
        t, inv = rn(y / s), rn(1 / s)
        q = rn(y * inv)
        without += q != t
        assert rn(q - rn(q * s - y) * inv) == t, (int(y), int(s))
        tried += 1
    assert tried > 1000 and without > 500          # and without the step it is not
