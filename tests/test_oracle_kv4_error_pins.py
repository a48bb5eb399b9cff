"""How far a quantised value may be off (include/tva.h, "4-bit cache"): half a scale from
2^-14 on; below, where scales are the multiples n 2^-17, at most 7 * 2^-18."""
from fractions import Fraction as F

import numpy as np
import pytest

import oracle

UNIT = 2.0 ** -17


def _blocks(top):
    """A block for each largest magnitude `top`: it, and values down to 0 of both signs."""
    f = np.linspace(1.0, 0.0, 16) * np.where(np.arange(16) % 2, -1.0, 1.0)
    return np.asarray(top, dtype=np.float64)[:, None] * f


def _off(x):
    byte, q = oracle.kv4_quantise(x)
    s = oracle.SCALES[byte]
    return np.abs(q * s - x).max(axis=1), s[:, 0], byte[:, 0]


def test_small_scales():
    """Largest magnitudes over every scale byte 0 .. 9 in steps of a 64th of 7 UNIT."""
    off, s, byte = _off(_blocks(np.arange(0, 9 * 64) / 64.0 * 7 * UNIT))
    assert set(byte) == set(range(10))
    assert (off[byte < 8] <= 7 * 2.0 ** -18).all() and (off[byte >= 8] <= s[byte >= 8] / 2).all()
    # the bound is met: just below the border between two scales
    assert off[byte < 8].max() >= 0.96 * 7 * 2.0 ** -18


@pytest.mark.parametrize("n,tops,scales_off", [(1, 10.4, 3.4), (2, 17.4, 1.7), (3, 24.4, 3.4 / 3)])
def test_half_a_scale_is_no_bound_for_small_scales(n, tops, scales_off):
    off, s, byte = _off(_blocks([tops * UNIT]))
    assert byte[0] == n and abs(off[0] / s[0] - scales_off) < 1e-9 and off[0] > s[0] / 2
    assert scales_off <= 3.5 / n


def test_normal_scales():
    """Every normal scale, largest magnitudes at and next to its borders: exact in float64."""
    lo = (oracle.SCALES[8:-1] + oracle.SCALES[7:-2]) * 3.5
    hi = (oracle.SCALES[8:-1] + oracle.SCALES[9:]) * 3.5
    for top in (lo, np.nextafter(lo, np.inf), np.nextafter(hi, 0), hi, (lo + hi) / 2):
        off, s, byte = _off(_blocks(top))
        keep = byte >= 8
        assert (off[keep] <= s[keep] / 2).all() and keep.sum() >= 200


def test_zero_and_saturation():
    off, s, byte = _off(_blocks([7 * 2.0 ** -18, np.nextafter(7 * 2.0 ** -18, 1), 7.5 * 2560, 7.6 * 2560]))
    assert list(byte) == [0, 1, 210, 210]
    assert F(float(off[0])) == 7 * F(1, 2 ** 18) and off[2] <= 1280 and off[3] > 1280
