"""lora_rotary_turns against whole-number arithmetic (no launches): the nearest 64-bit
fraction of a turn of any finite frequency."""
import ctypes
import math
import random
from fractions import Fraction

import pytest

import test_block_ops_abi_cpu as abi
from rank_linear_gb300 import _lib

PLACES = 1400


def setup_module():
    abi.setup_module()


def arctan_of_one_over(n, one):
    """one * atan(1 / n) by its series."""
    total = term = one // n
    k, sign = 1, 1
    while term:
        term //= n * n
        k, sign = k + 2, -sign
        total += sign * (term // k)
    return total


def over_two_pi():
    """1 / (2 pi) as a fraction, good to 2^-1350: pi = 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << PLACES
    pi = 16 * arctan_of_one_over(5, one) - 4 * arctan_of_one_over(239, one)
    assert abs(pi / one - math.pi) < 1e-15
    return Fraction(one, 2 * pi)


def turns(values):
    out = (ctypes.c_uint64 * len(values))()
    assert abi.L.lora_rotary_turns((ctypes.c_double * len(values))(*values), len(values), out) == _lib.LORA_OK
    return list(out)


def frequencies():
    w = [1.0, -1.0, 0.5, 2 * math.pi, math.pi, -2 * math.pi, 100.0, 1e-9, 0.0, -0.0, 1e15, 2.0 ** 53, 2.0 ** 200,
         1.7e308, -1.7e308, 5e-324, 2.0 ** -64, 1e-18, 3e-20, 6.283185307179587e-19]
    w += [500000.0 ** (-2 * i / 128) / f for i in range(64) for f in (1.0, 4.0, 16.0)]
    r = random.Random(1)
    return w + [math.ldexp(r.uniform(-1, 1), r.randint(-80, 1000)) for _ in range(500)]


def test_every_frequency_to_the_nearest():
    c, w = over_two_pi(), frequencies()
    for x, t in zip(w, turns(w)):
        exact = Fraction(x) * c * 2 ** 64 % 2 ** 64
        off = abs(Fraction(t) - exact)
        off = min(off, 2 ** 64 - off)
        assert off <= Fraction(1, 2) + Fraction(1, 1024), (x, float(off))


@pytest.mark.parametrize("x", [1.0, 0.3, 123.456])
def test_negative_frequencies_turn_the_other_way(x):
    a, b = turns([x, -x])
    assert (a + b) % 2 ** 64 == 0
