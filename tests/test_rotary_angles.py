"""Cosine and sine of the rotation: the kernels' steps in float32, done in numpy,
against float64.

A fraction of a turn is cut to 2^-34 turns (2^-31.3 of an angle) and to the
nearest quarter; the rest x, |x| <= pi / 4, carries the roundings of the integer,
of the constant and of their product, 3 * 2^-24 pi / 4 in all: 2^-22.8.  The first
terms left out are 1.8e-9 (x^11 / 11!) and 2.5e-8 (x^10 / 10!), and the last
steps of the sums round values up to 1, 2^-25, after terms that are at most x^2 / 2 <
0.31 with under 4 roundings of their own, 0.31 * 4 * 2^-25.  Together 1.4e-7 + 2.5e-8 +
3e-8 + 3.7e-8 < 2.4e-7 = 2^-22, and with the product by mscale, 2^-25 of it and its own
rounding, under 2^-21: the bound that the tests of rotated values use."""
import math
import random

import numpy as np
import pytest

f32 = np.float32
TOP = 1 << 64


def fma(a, b, c):
    return f32(np.float64(a) * np.float64(b) + np.float64(c))


def cos_sin(pos, freq):
    turn = pos * freq % TOP
    quarter = (turn + (1 << 61)) % TOP >> 62
    rest = turn >> 30 & 0xffffffff
    x = f32(f32(rest - (1 << 32) if rest >> 31 else rest) * f32(3.6572954e-10))
    y = f32(x * x)
    sn = fma(y, f32(1 / 362880), f32(-1 / 5040))
    sn = fma(y, sn, f32(1 / 120))
    sn = fma(y, sn, f32(-1 / 6))
    sn = fma(f32(x * y), sn, x)
    cs = fma(y, f32(1 / 40320), f32(-1 / 720))
    cs = fma(y, cs, f32(1 / 24))
    cs = fma(y, cs, f32(-0.5))
    cs = fma(y, cs, f32(1))
    return [(cs, sn), (-sn, cs), (-cs, -sn), (sn, -cs)][quarter]


def exact(pos, freq):
    turn = pos * freq % TOP
    eighths, rest = turn >> 61, turn & (1 << 61) - 1                # to keep all bits of the angle
    a = math.pi / 4 * (rest / 2 ** 61)
    b = math.pi / 4 * eighths
    return (math.cos(a) * math.cos(b) - math.sin(a) * math.sin(b),
            math.sin(a) * math.cos(b) + math.cos(a) * math.sin(b))


@pytest.mark.parametrize("far", [1, 1 << 10, 1 << 20, (1 << 31) - 1])
def test_cos_sin(far):
    rng = random.Random(far)
    worst = 0.0
    for i in range(6000):
        pos, freq = rng.randint(-far, far), rng.randrange(TOP)
        if i % 3 == 0:                                              # next to the eighths of a turn
            pos, freq = 1, (rng.randrange(8) << 61) + rng.randint(-3, 3) * rng.choice((1, 1 << 29, 1 << 40))
        got, want = cos_sin(pos, freq % TOP), exact(pos, freq % TOP)
        worst = max(worst, *(abs(float(g) - w) for g, w in zip(got, want)))
    assert worst <= 2.0 ** -22, worst
