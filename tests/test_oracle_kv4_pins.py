"""The 4-bit record's oracle against its definition in exact fractions."""
from fractions import Fraction as F

import numpy as np
import pytest

import oracle


def _scale(byte):
    return F(byte, 2 ** 17) if byte < 8 else F(8 + byte % 8) * F(2) ** (byte // 8 - 18)


def _nearest_scale(x):
    """By trying all of them; a tie goes to the even byte."""
    best = min(range(211), key=lambda b: (abs(_scale(b) - x), b % 2))
    return best


def _nearest_whole(x):
    lo = x.numerator // x.denominator
    return min((lo, lo + 1), key=lambda q: (abs(x - q), q % 2))


def test_scales_are_the_format():
    assert [F(float(s)) for s in oracle.SCALES] == [_scale(b) for b in range(211)]
    assert oracle.SCALES[210] == 2560 and oracle.SCALES[8] == 2.0 ** -14
    # shifted left by 7 a byte is the same value in float16
    half = (np.arange(211, dtype=np.uint16) << 7).view(np.float16)
    assert np.array_equal(half.astype(np.float64), oracle.SCALES)


@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32", "tiny", "borders", "huge"])
def test_quantise_is_the_definition_in_fractions(kind):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((40, 16)) * 2.0 ** rng.integers(-12, 6, (40, 1))).astype(np.float32)
    if kind == "bf16":
        x = (x.view(np.uint32) & np.uint32(0xffff0000)).view(np.float32)
    elif kind == "fp16":
        x = x.astype(np.float16).astype(np.float32)
    elif kind == "tiny":
        x = (x * 2.0 ** -14).astype(np.float32)
    elif kind == "borders":  # halves of a scale, and 7 (8 + m + 1/2): ties of both roundings
        x = (rng.integers(-15, 16, (40, 16)) * 0.5 * 2.0 ** -3 * rng.integers(8, 16, (40, 1))).astype(np.float32)
        x[:20, 0] = 7 * (rng.integers(8, 16, 20) + 0.5)
    elif kind == "huge":
        x = (x * 2.0 ** 14).astype(np.float32)
    byte, q = oracle.kv4_quantise(x)
    for i in range(40):
        top = max(abs(F(float(v))) for v in x[i])
        b = _nearest_scale(top / 7)
        assert int(byte[i, 0]) == b
        for e in range(16):
            want = 0 if b == 0 else max(-7, min(7, _nearest_whole(F(float(x[i, e])) / _scale(b))))
            assert int(q[i, e]) == want


def test_nan_infinity_and_zero_blocks():
    x = np.zeros((4, 16))
    x[1, 3], x[1, 4] = np.nan, 3.5
    x[2, 0], x[2, 1], x[2, 2] = np.inf, -np.inf, 1.0
    x[3] = 7 * 2.0 ** -18  # the largest that becomes 0: a tie with scale byte 1
    byte, q = oracle.kv4_quantise(x)
    assert list(byte[:, 0]) == [0, 104 + 8, 210, 0]
    assert q[1, 3] == 0 and q[1, 4] == 7 and list(q[2, :3]) == [7, -7, 0] and not q[3].any()


@pytest.mark.parametrize("d,size", [(64, 80), (128, 144)])
def test_pack_and_unpack(d, size):
    rng = np.random.default_rng(6)
    k, v = rng.standard_normal((2, 5, 3, d))
    rec = oracle.kv4_pack(k, v)
    assert rec.shape == (5, 3, size) and oracle.kv4_record_bytes(d) == size
    for x, (byte, q) in zip((k, v), oracle.kv4_unpack(rec, d)):
        b, w = oracle.kv4_quantise(x)
        assert np.array_equal(b, byte) and np.array_equal(w, q)
    K, V = oracle.kv4_values(rec, d)
    s = np.repeat(oracle.SCALES[oracle.kv4_quantise(k)[0]], 16, axis=-1)
    assert (np.abs(K - k) <= s / 2 + 1e-12).all()
    # the layout, byte by byte: element 8 i + e of K
    for e in range(8):
        bit = 4 * (e // 2) + 16 * (e % 2)
        nib = (rec[:, :, bit // 8:d // 2:4] >> (bit % 8)) & 15
        assert np.array_equal(nib.astype(int) - 8, oracle.kv4_quantise(k)[1][:, :, e::8])
    # a second rounding changes nothing
    assert np.array_equal(oracle.kv4_pack(K, V), rec)
    # every value is exact in bfloat16 and float16
    for x in (K, V):
        assert np.array_equal(x.astype(np.float16).astype(np.float64), x)
        assert not (x.astype(np.float32).view(np.uint32) & 0xffff).any()
