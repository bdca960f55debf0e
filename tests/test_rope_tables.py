"""The frequency tables of the scaling by index against numbers worked out apart (no GPU): 50-digit decimal arithmetic from
the definition, f_i = base^(-2 i / rot), s falling from 1 at the index of `high` turns (rounded down) to 0 at that of `low`
turns (rounded up), f_i (s + (1 - s) / factor). Where the slowest frequency turns more than `low` times in the original
context, the ramp ends beyond the last index and no frequency is divided by all of the factor."""
import math

import numpy as np
import pytest

import fp8_weight_only_skinny_gb300 as sk
from oracle import rope

# rot, base, original, factor, low: {index: radians per position}
TABLES = [
    # ramp 45 .. 70; the last index, 63, turns 2.409 times
    ((128, 10000.0, 131072, 4.0, 1.0), {44: 1.778279410038922801e-3, 45: 1.539926526059491990e-3, 46: 1.293515789198424305e-3,
                                        50: 6.374100779325874532e-4, 57: 1.752588565929191228e-4, 62: 6.534255017600287726e-5,
                                        63: 5.311997129571507626e-5}),
    # ramp 40 .. 65; 1.204 times
    ((128, 10000.0, 65536, 8.0, 1.0), {39: 3.651741272548377058e-3, 40: 3.162277660168379332e-3, 52: 3.261579686104024666e-4,
                                       63: 2.251824870144443450e-5}),
    # ramp 24 .. 37; 5.564 times
    ((64, 10000.0, 262144, 2.0, 1.0), {25: 7.210521243581306032e-4, 26: 5.190843001757068434e-4, 28: 2.675773404757859435e-4,
                                       31: 9.744964311962752495e-5}),
    # ramp 11 .. 23; 3.710 times
    ((32, 10000.0, 131072, 4.0, 0.0625), {0: 1.0, 12: 9.375e-4, 15: 1.333709557529192101e-4}),
    # ramp 23 .. 40, within the table
    ((128, 1000000.0, 32768, 8.0, 1.0), {24: 5.333972863937869954e-3, 30: 9.851000571115867874e-4, 39: 3.894236592502217295e-5,
                                         40: 2.222849262548653502e-5, 63: 1.551172200939649458e-7}),
]


@pytest.mark.parametrize("args,want", TABLES)
def test_numbers_worked_out_apart(args, want):
    rot, base, original, factor, low = args
    got = sk.rope_frequencies(rot, base, "index", factor=factor, original=original, low=low, high=32.0, device="cpu").numpy()
    ref = rope.frequencies(rot, base, "index", factor=factor, original=original, low=low, high=32.0)
    for i, f in want.items():
        # a few operations in double precision, then cut to a whole number
        assert abs(int(got[i]) * 2.0 ** -64 * 2 * math.pi - f) <= 2.0 ** -44 * f + 2.0 ** -60
        assert abs(ref[i] - f) <= 2.0 ** -44 * f


@pytest.mark.parametrize("rot", [16, 64, 128, 256])
@pytest.mark.parametrize("original", [1024, 32768, 131072, 4194304, 10 ** 12])
@pytest.mark.parametrize("low,high", [(1.0, 32.0), (0.5, 50.0)])
def test_only_frequencies_that_turn_seldom_are_divided_by_all_of_the_factor(rot, original, low, high):
    factor = 4.0
    got = sk.rope_frequencies(rot, 10000.0, "index", factor=factor, original=original, low=low, high=high, device="cpu").numpy()
    kept = got * 2.0 ** -64 / (10000.0 ** (-2.0 * np.arange(rot // 2) / rot) / (2 * math.pi))
    turns = original * 10000.0 ** (-2.0 * np.arange(rot // 2) / rot) / (2 * math.pi)
    assert np.all(kept[turns > high * (1 + 1e-9)] > 1 / factor + 1e-3)
    assert np.all(np.diff(kept) < 1e-9) and np.all(kept < 1 + 1e-9) and np.all(kept > 1 / factor - 1e-9)
    step = 10000.0 ** (2.0 / rot)                              # one index on, a frequency turns so much less
    assert np.all(kept[turns > low * (1 + 1e-9)] > 1 / factor + 1e-9)
    assert np.allclose(kept[turns < low / step], 1 / factor, rtol=1e-9)
