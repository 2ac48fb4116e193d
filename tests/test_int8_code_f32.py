"""The 8-bit code of an fp32 value by one fma (int8.cuh), as the few-token layer codes its hidden rows: the exact code, or the
one above in size when the quotient lies below a half-integer by less than 2^-23 of itself."""
from fractions import Fraction

import numpy as np

MAGIC = Fraction(12582912)  # 1.5 * 2^23: adding it rounds to an integer, ties to even


def inverse_up(a):
    """127 / a in fp32, rounded up."""
    want = Fraction(127) / Fraction(float(a))
    inv = np.float32(127.0) / a
    if Fraction(float(inv)) < want:
        inv = np.nextafter(inv, np.float32(np.inf))
    assert Fraction(float(np.nextafter(inv, np.float32(0)))) < want <= Fraction(float(inv))
    return inv


def fma_code(v, inv):
    """fma(v, inv, magic) - magic: the sum lies in [2^23, 2^24), where fp32 holds the integers, and is rounded once."""
    return int(round(Fraction(float(v)) * Fraction(float(inv)) + MAGIC) - MAGIC)


def test_code_of_fp32_values():
    rng = np.random.default_rng(4)
    above = 0
    for _ in range(400):
        a = np.float32(rng.uniform(1, 2) * 2.0 ** rng.integers(-60, 60))
        inv = inverse_up(a)
        assert fma_code(a, inv) == 127 and fma_code(-a, inv) == -127
        # values anywhere, and the fp32 values around the half-integer quotients
        v = [np.float32(x) for x in rng.uniform(-1, 1, 20) * a]
        for o in rng.integers(0, 127, 10):
            h = np.float32((int(o) + 0.5) / 127 * float(a))
            v += [np.nextafter(h, np.float32(0)), h, np.nextafter(h, np.float32(np.inf)), -h]
        for x in v:
            q = Fraction(127) * Fraction(float(x)) / Fraction(float(a))
            if abs(q) > 127:
                continue
            got, exact = fma_code(x, inv), int(round(q))  # round(): ties to even
            if got != exact:
                half = Fraction(2 * abs(exact) + 1, 2)
                assert abs(got) == abs(exact) + 1 and 0 <= half - abs(q) < abs(q) * Fraction(1, 2 ** 23), (a, x)
                above += 1
    assert above > 0  # the rule does meet such values
