"""The 8-bit code of a bf16 value without a division (int8.cuh): one fma of the value with 127 / a rounded up, on every
pair of 8-bit significands and exponent distance, against exact rationals."""
from fractions import Fraction

import numpy as np


def test_one_fma_gives_the_exact_code():
    magic = 12582912.0  # 1.5 * 2^23: adding it in fp32 rounds to an integer, ties to even
    for A in range(128, 256):
        want = Fraction(127, A)
        inv = np.float32(127.0 / A)
        if Fraction(float(inv)) < want:  # rounded up
            inv = np.nextafter(inv, np.float32(np.inf))
        assert Fraction(float(np.nextafter(inv, np.float32(0)))) < want <= Fraction(float(inv))
        for e in range(12):
            v = np.arange(128, 256) * 2.0 ** -e
            v = v[v <= A]
            # 8 + 24 significant bits: the product and its sum with the magic number are exact in 64 bits, and the
            # conversion to 32 bits is the fma's one rounding
            code = (v * float(inv) + magic).astype(np.float32) - np.float32(magic)
            exact = [int(round(Fraction(float(x)) * 127 / A)) for x in v]  # round(): ties to even
            assert code.astype(int).tolist() == exact, (A, e)
