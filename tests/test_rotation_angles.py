"""The steps that form a rotation's cosines, against whole-number arithmetic."""
import math

import numpy as np

import angles_ref as A


def test_the_reference():
    for p, f in ((0, 1.0), (1, 1.0), (-3, 0.5), (1000, 0.37), (2 ** 20, 1.0)):
        c, s = A.exact(p, f)
        assert math.isclose(c, math.cos(p * f), abs_tol=1e-9) and math.isclose(s, math.sin(p * f), abs_tol=1e-9)
    # the nearest fp64 number to 355/113 turns' worth of a far multiple of pi: sine of n pi is 0
    n = 10 ** 9
    assert abs(A.exact(1, n * math.pi)[1]) < n * 2.0 ** -52


def test_cosines_are_as_good_as_stated():
    """2^-22 for angles up to 2^28, 2^-20 up to 2^31: positions of every size, of both signs."""
    rng = np.random.default_rng(5)
    worst = {}
    for top in (1, 2 ** 10, 2 ** 20, 2 ** 27, 2 ** 28, 2 ** 29, 2 ** 31 - 1):
        pos = rng.integers(max(1, top // 2), top + 1, 3000) * rng.choice([-1, 1], 3000)
        freq = rng.choice([1.0, 0.7498942093324559, 500000.0 ** -0.03125, 0.999], 3000) * rng.choice([1.0, 1.0 - 2.0 ** -30], 3000)
        c, s = A.steps(pos, freq)
        off = 0.0
        for i in range(len(pos)):
            ec, es = A.exact(pos[i], freq[i])
            d = max(abs(float(c[i]) - ec), abs(float(s[i]) - es))
            assert d <= A.error(pos[i] * freq[i]), (pos[i], freq[i], math.log2(d))
            off = max(off, d)
        worst[top] = math.log2(off)
    # and it does not hold beyond: the larger figure of the last range is needed
    assert worst[2 ** 31 - 1] > -22, worst


def test_all_octants():
    """Angles around the borders of the reduction, at small positions and far ones."""
    pos, freq = [], []
    for k in range(-16, 17):
        for p in (1, 3, 2 ** 16 + 1):
            for d in (-1e-7, 0.0, 1e-7):
                pos.append(p)
                freq.append((k * math.pi / 4 + d) / p)
    pos, freq = np.array(pos), np.array(freq)
    c, s = A.steps(pos, freq)
    for i in range(len(pos)):
        ec, es = A.exact(pos[i], freq[i])
        assert max(abs(float(c[i]) - ec), abs(float(s[i]) - es)) <= 2.0 ** -22
