"""Cosines and sines of position * freq from whole-number arithmetic with 60 digits of pi, and
the rotation's own steps in numpy."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np

PI = Fraction(3141592653589793238462643383279502884197169399375105820974944, 10 ** 60)


def exact(position: int, freq: float):
    """(cos, sin) of the real number position * freq, to fp64 rounding."""
    angle = int(position) * Fraction(*float(freq).as_integer_ratio())
    left = float(angle - 2 * PI * round(angle / (2 * PI)))
    return math.cos(left), math.sin(left)


def steps(positions, freqs):
    """(cos, sin) as the kernel forms them: turns and their reduction in fp64, polynomials over an
    eighth of a turn in fp32 (a fused operation is one rounding of an fp64 value)."""
    f32 = np.float32
    turns = positions.astype(np.float64) * (freqs.astype(np.float64) * 0.15915494309189535)
    part = turns - np.rint(turns)
    quarter = np.rint(4.0 * part)
    x = ((part - 0.25 * quarter) * 6.283185307179586).astype(f32)
    fma = lambda a, b, c: (a.astype(np.float64) * b.astype(np.float64) + np.asarray(c, f32).astype(np.float64)).astype(f32)  # noqa: E731
    t = x * x
    one = lambda d: f32(1) / f32(d)  # noqa: E731
    p = fma(t, np.full_like(t, one(362880)), -one(5040))
    p = fma(t, fma(t, p, one(120)), -one(6))
    s = fma(x * t, p, x)
    p = fma(t, np.full_like(t, one(40320)), -one(720))
    p = fma(t, fma(t, p, one(24)), f32(-0.5))
    c = fma(t, p, f32(1))
    q = quarter.astype(np.int64)
    cos, sin = np.where(q & 1, s, c), np.where(q & 1, c, s)
    return np.where((q + 1) & 2, -cos, cos), np.where(q & 2, -sin, sin)


# What a cosine may be off by. fp64: the constant 1 / 2 pi, its product with freq and that with
# the position are rounded, 3 * 2^-53 of the angle at most: 2^-23.4 at 2^28, 2^-20.4 at 2^31.
# fp32, of values up to 1: the reduced angle (2^-25, times a sine below 0.71), its square (2^-25.7),
# the polynomial's end (2^-25.3) and last addition (2^-25), the rest below 2^-27: 2^-23.2 together.
ERROR = ((2 ** 28, 2.0 ** -22), (2 ** 31, 2.0 ** -20))


def error(angle: float) -> float:
    return next(e for most, e in ERROR if abs(angle) <= most)
