"""The factor of a key's norm is the fp32 value next to the exact one: rows whose squares lie as far as they can
from what the kernel adds up exactly, with factors just beside the middle of two fp32 values.

The kernel cuts each square at multiples of 2^-9 (for a sum in [2^7, 2^8)) and adds the parts apart. Values
here are multiples of 2^-14 near 1, so the rests are multiples of 2^-28 below 2^-10 and a lane's sums of
them exact; the lanes' sums, below 2^-3, are off by less than 2^-26 in all, 2^-34 of the factor. One step of
Newton from a factor that is off by 2^-22 leaves far less. So a factor that lies 2^-10 of the distance of two
fp32 values (2^-34 of itself, where its mantissa is near 2) or more beside their middle is rounded to its own side."""
from fractions import Fraction
from math import isqrt

import numpy as np
import pytest
import torch

from gpu_util import to_dev_i32
from speculative_decoding_verification_w12_gb300 import w12

pytestmark = pytest.mark.gpu
EPS = np.float32(1e-11)


def _beside(units, above):
    """(nearest fp32 factor, how far from the middle of two, in their distance) of a row of 128 values
    units 2^-14, with the factor above (below) the middle; None otherwise."""
    m = Fraction(int((units * units).sum()), 128 << 28) + Fraction(float(EPS))
    scale = 1 << 120
    r = Fraction(isqrt(m.denominator * scale * scale // m.numerator), scale)       # to 2^-119
    if not Fraction(1, 2) <= r < 1:
        return None
    steps = r * (1 << 24)                                                          # fp32 values are 2^-24 apart here
    low = int(steps)
    off = steps - low - Fraction(1, 2)
    if (off > 0) != above:
        return None
    return np.float32((low + above) / 2.0 ** 24), abs(float(off))


def _rows(above, n):
    """Rows whose rests have one sign, their factors 2^-10 to 2^-8.5 of the distance beside the middle."""
    g = np.random.default_rng(int(above))
    k = np.arange(1, 700)
    rest = ((2 * k * 2.0 ** -14 + k * k * 2.0 ** -28) * 2.0 ** 9) % 1.0
    # A rest above a half is a square's way up to the next multiple: the sum of the cut parts is too high.
    some = k[(rest > 0.52) & (rest < 0.56)] if above else k[(rest > 0.44) & (rest < 0.48)]
    rows, want = [], []
    while len(rows) < n:
        units = 16384 + g.choice(some, 128)
        f = _beside(units.astype(object), above)
        if f and 2.0 ** -10 <= f[1] <= 2.0 ** -8.5:
            rows.append(units * 2.0 ** -14)
            want.append(f[0])
    return np.array(rows, dtype=np.float32), np.array(want)


@pytest.mark.parametrize("above", [False, True])
def test_factors_beside_the_middle_of_two(above):
    x, f = _rows(above, 40)
    tab = np.concatenate([np.ones((1, 64)), np.zeros((1, 64))], 1).astype(np.float32)   # no turn
    one = torch.ones(128, device="cuda")
    rope = w12.Rope(torch.from_numpy(tab).cuda(), 128, one, one, float(EPS))
    got = rope.run(None, torch.from_numpy(x[:, None]).cuda(), to_dev_i32(np.zeros(len(x))), dtype=torch.float32)[1].cpu().numpy()[:, 0]
    wrong = [i for i in range(len(x)) if not np.array_equal(got[i], x[i] * f[i])]
    assert not wrong
