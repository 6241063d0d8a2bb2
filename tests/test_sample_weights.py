"""Host model of the sampler's integer weights: weight_bits() of sampling.cuh restated in exact rational arithmetic,
rounded where the kernel rounds.  It forms an exponent by adding to a word, so it is right only down to the logit
below which weights count as 0; the model checks that this bound, rounded up to float32, keeps every weight right, and
that rounded down it would not."""
import math
import struct
from fractions import Fraction

import numpy as np
import pytest

LN2 = math.log(2.0)


def fma(a, b, c):
    return float(Fraction(a) * Fraction(b) + Fraction(c))


def bits(x):
    return struct.unpack("<Q", struct.pack("<d", x))[0]


def weight(x, m, T, fx):
    """The weight of logit x as the kernel computes it, in units of 2^-fx, modulo 2^64."""
    a = [LN2 / 32]
    for i in range(2, 6):
        a.append(a[-1] * a[0] / i)
    c32, shift, magic = (1 / T) * (32 / LN2), 1.5 * 2.0 ** 52, 2.0 ** (52 - fx)
    d = float(x) - float(m)
    t = fma(d, c32, shift)
    r = fma(d, c32, shift - t)
    p = 0.0
    for c in a[::-1]:
        p = fma(p, r, c)
    p = fma(p, r, 1.0)
    n = bits(t) & 0xffffffff
    n -= (n >> 31) << 32
    e = bits(2.0 ** ((n & 31) / 32))
    e = (((e >> 32) + (n >> 5) * 2 ** 20) & 0xffffffff) << 32 | (e & 0xffffffff)
    return (bits(fma(struct.unpack("<d", struct.pack("<Q", e))[0], p, magic)) - bits(magic)) % 2 ** 64


def bound(m, T, fx, up):
    """The smallest logit with a weight, as a float32."""
    exact = float(m) - (fx + 2) * LN2 * T
    y = np.float32(exact)
    if up and float(y) < exact:
        y = np.nextafter(y, np.float32(np.inf))
    if not up and float(y) > exact:
        y = np.nextafter(y, np.float32(-np.inf))
    return y


def right(x, m, T, fx):
    # rounding to an integer, and a relative error below 2^-45 of the exponential
    want = 2.0 ** fx * math.exp((float(x) - float(m)) / T)
    return abs(weight(x, m, T, fx) - want) <= 0.5 + 2.0 ** -45 * want


CASES = [(10.0, 1e-9), (1e4, 1e-6), (1e10, 1.0), (-3e38, 3.4e29), (2.0, 2e-9), (0.0, 1e-38), (1e-30, 1e-38),
         (3e38, 1e30), (-5.0, 0.7), (12.0, 50.0)]


@pytest.mark.parametrize("fx", [43, 45, 48])
@pytest.mark.parametrize("m,T", CASES)
def test_weights_from_the_bound_on_are_right(m, T, fx):
    m, T = np.float32(m), float(np.float32(T))
    least = bound(m, T, fx, True)
    assert least <= m and weight(m, m, T, fx) == 2 ** fx
    x = [m]
    for _ in range(8):
        x.append(np.nextafter(x[-1], np.float32(-np.inf)))
    x += list(np.linspace(least, m, 50, dtype=np.float64).astype(np.float32)) + [least]
    for v in x:
        if least <= v <= m:
            assert right(v, m, T, fx), v
        elif v < least:  # what is left out weighs less than the sums resolve
            assert math.exp((float(v) - float(m)) / T) < 2.0 ** -(fx + 1)


@pytest.mark.parametrize("m,T", [(10.0, 1e-9), (1e4, 1e-6), (1e10, 1.0)])
def test_the_bound_rounded_down_would_admit_a_wrong_weight(m, T):
    m, T = np.float32(m), float(np.float32(T))
    v = bound(m, T, 45, False)
    assert v < m and not right(v, m, T, 45) and weight(v, m, T, 45) > 2 ** 45
