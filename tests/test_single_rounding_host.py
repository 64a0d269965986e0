"""The reference of one-rounding sums against exact fractions."""
import random
import struct
from fractions import Fraction

import numpy as np
import torch

from single_rounding import fma


def _f32(rng, lo=100, hi=150):
    return struct.unpack("f", struct.pack("I", rng.getrandbits(23) | rng.randint(lo, hi) << 23 | rng.getrandbits(1) << 31))[0]


def test_one_rounding():
    """The nearest fp32 value, the even one of two: for random values, and for
    sums next to the middle of two, where 64 bits alone would round twice."""
    rng = random.Random(1)
    cases = []
    for _ in range(4000):
        a, b = _f32(rng), _f32(rng)
        cases.append((a, b, float(np.float32(rng.choice([_f32(rng), a * b * rng.choice([1, -1, 2.0 ** 24, 2.0 ** 30])])))))
    for _ in range(200):  # 1 + 2^-24 (the middle) and a bit far below
        tiny = 2.0 ** -rng.randint(25, 60)
        cases.append((2.0 ** -24, float(np.float32(1 + rng.choice([-1, 1]) * 2.0 ** -rng.randint(20, 24))), 1.0))
        cases.append((tiny, 2.0 ** -rng.randint(1, 20), float(np.float32(1 + 2.0 ** -23))))
    a, b, c = (torch.tensor(v) for v in zip(*cases))
    got = fma(a, b, c).numpy()
    for (x, y, z), g in zip(cases, got):
        want = Fraction(x) * Fraction(y) + Fraction(z)
        off = abs(Fraction(float(g)) - want)
        for side in (np.nextafter(g, np.float32(np.inf)), np.nextafter(g, np.float32(-np.inf))):
            other = abs(Fraction(float(side)) - want)
            assert off < other or (off == other and g.view(np.uint32) & 1 == 0), (x, y, z, g)
