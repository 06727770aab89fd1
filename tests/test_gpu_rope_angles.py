"""The angle of idx_rope_append at positions up to 2^31 - 1, against whole numbers.

The reference forms position * inv_freq / (2 pi) modulo 1 with 256 bits.  A
pair (1, 0) in fp32 comes back as the cosine and sine of what the kernel makes
of it.  Bound: the angle within 2^-33 turns; its fraction h of a half turn as
fp32 (relative 2^-24: pi |h| 2^-24 radians); sine and cosine within 2 units in
the last place and two roundings, 4 * 2^-24 of the value.
"""

import math
from fractions import Fraction

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BITS = 256


def inverse_two_pi():
    """2^BITS / (2 pi), pi by Machin's formula 16 atan(1/5) - 4 atan(1/239)."""
    one = 1 << (BITS + 64)

    def atan_inverse(n):
        total, term, k, sign = 0, one // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return total

    pi = 16 * atan_inverse(5) - 4 * atan_inverse(239)
    return (1 << BITS) * one // (2 * pi)


def turns(freq, position, inv):
    """The angle in turns, in [-1/2, 1/2)."""
    f = Fraction(float(freq)) * position * inv / (1 << BITS)
    f -= math.floor(f)
    return float(f if f < Fraction(1, 2) else f - 1)


def test_inverse_two_pi():
    assert abs(inverse_two_pi() / 2**BITS - 1 / (2 * math.pi)) < 2.0**-54


@pytest.mark.parametrize("dim", [8, 2])  # rows of whole pieces, and pairs apart
@pytest.mark.parametrize("base", [10000.0, 500000.0, 1000000.0])
def test_far_angles(lib, base, dim):
    inv = inverse_two_pi()
    f, _ = lib.idx_rope_frequencies(128, base)
    pos = torch.arange(2**31 - 1 - 1500, 2**31 - 1, dtype=torch.int64).to(torch.int32)
    x = torch.zeros(len(pos), 1, dim, device="cuda")
    half = dim // 2
    x[..., :half] = 1.0
    worst = 0.0
    for lo in range(0, 16, half):  # the fastest frequencies lose most
        freq = f[lo : lo + half]
        y = torch.empty_like(x)
        lib.idx_rope_append(x, None, None, pos.cuda(), freq.cuda(), y, None, None)
        got = y.double().cpu().numpy()[:, 0]
        t = np.array([[turns(w, p, inv) for w in freq.tolist()] for p in pos.tolist()])
        a = 2 * math.pi * t
        slack = 2 * math.pi * 2.0**-33 + math.pi * np.abs(2 * t) * 2.0**-24
        for at, want in ((got[:, :half], np.cos(a)), (got[:, half:], np.sin(a))):
            worst = max(worst, float((np.abs(at - want) - slack - 4 * 2.0**-24 * np.abs(want)).max()))
    assert worst <= 0, worst
