"""The 64-bit exponential of the routing kernels, its steps done in exact arithmetic with each rounding applied: the constants
are what their comment says, and the error is within the 2^-46 that it states."""
import math
import os
import random
import re
from fractions import Fraction

import tiled_dense_gemm_bias_amd as gba

SOURCE = os.path.join(os.path.dirname(os.path.abspath(gba.__file__)), "csrc", "moe", "gm_route.hpp")


def ln2(bits=200):
    """sum of 1 / (i 2^i), to well below 2^-bits."""
    return sum(Fraction(1, i << i) for i in range(1, bits))


def exp(d):
    """e^d of a rational d, |d| <= 1, to below 2^-90."""
    term, total = Fraction(1), Fraction(0)
    for i in range(1, 30):
        total, term = total + term, term * d / i
    return total


def constants():
    text = open(SOURCE).read()
    hi, lo = re.search(r"kLn2 = ([0-9.e-]+), kLn2Rest = ([0-9.e-]+);", text).groups()
    body = text[text.index("double exp_neg(double d)"):]
    body = body[:body.index("\n}")]
    return float(hi), float(lo), body


def test_ln2_in_two_numbers():
    hi, lo, body = constants()
    assert hi == float(ln2()) and lo == float(ln2() - Fraction(hi))
    assert "fma(n, -kLn2Rest, fma(n, -kLn2, c))" in body
    assert len(re.findall(r"1\.0 / \d+\.0", body)) == 9                          # 1 / 3! .. 1 / 11!
    assert [int(n) for n in re.findall(r"1\.0 / (\d+)\.0", body)] == [math.factorial(i) for i in (11, 10, 9, 8, 7, 6, 5, 4, 3)]


def test_within_2_to_the_minus_46():
    hi, lo, _ = constants()

    def fma(a, b, c):
        return float(Fraction(a) * Fraction(b) + Fraction(c))
    rng = random.Random(3)
    worst = 0.0
    for i in range(500):
        d = -rng.random() * rng.choice([1e-3, 1, 30, 700]) if i else -0.0
        if i % 5 == 1:
            d = float(-(rng.randint(0, 900) + Fraction(1, 2)) * ln2())           # r at its largest
        n = float(round(Fraction(d * 1.4426950408889634)))
        r = fma(n, -lo, fma(n, -hi, d))
        p = fma(1.0 / math.factorial(11), r, 1.0 / math.factorial(10))
        for k in (9, 8, 7, 6, 5, 4, 3):
            p = fma(p, r, 1.0 / math.factorial(k))
        for c in (0.5, 1.0, 1.0):
            p = fma(p, r, c)
        want = exp(Fraction(d) - int(n) * ln2())
        worst = max(worst, abs(float((Fraction(p) - want) / want)))
    assert worst < 2.0 ** -46
