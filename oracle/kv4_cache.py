"""The 4-bit K/V record: rounding, layout and values, in float64 and whole numbers.

TEST INFRASTRUCTURE ONLY (see the package docstring): never called by the library.

A block of 16 values x is stored as whole multiples q of a scale s: s is max |x| / 7
rounded to the nearest unsigned 5-exponent-bit, 3-mantissa-bit float (bias 15, subnormals,
at most 2560; ties to the even byte), and q is x / s rounded to the nearest whole number
(ties to even), within -7 .. 7.  NaN counts as 0; infinities saturate.
"""
from __future__ import annotations

import numpy as np

__all__ = ["SCALES", "kv4_quantise", "kv4_pack", "kv4_unpack", "kv4_values", "kv4_record_bytes"]

MAX_BYTE = 210
#: The scale bytes' values, ascending.
SCALES = np.array([b * 2.0 ** -17 if b < 8 else (8 + b % 8) * 2.0 ** (b // 8 - 18) for b in range(MAX_BYTE + 1)])


def kv4_record_bytes(d: int) -> int:
    return (9 * d // 8 + 15) // 16 * 16


def kv4_quantise(x):
    """(scale bytes [..., d / 16], multiples [..., d]) of x [..., d]."""
    x = np.asarray(x, dtype=np.float64)
    x = np.where(np.isnan(x), 0.0, x)
    blocks = x.reshape(*x.shape[:-1], -1, 16)
    top = np.abs(blocks).max(axis=-1)
    # max |x| against 7 (s_i + s_{i+1}) / 2: every border compared without a division
    border = (SCALES[1:] + SCALES[:-1]) * 3.5
    lo = np.searchsorted(border, top, side="left")
    hi = np.searchsorted(border, top, side="right")
    byte = np.where(lo == hi, lo, lo + lo % 2)  # on a border: the even one of lo, lo + 1
    s = SCALES[byte][..., None]
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(s > 0, np.clip(np.rint(np.where(s > 0, blocks / np.where(s > 0, s, 1), 0)), -7, 7), 0)
    return byte.astype(np.uint8), q.reshape(x.shape).astype(np.int64)


def kv4_pack(k, v):
    """Records [n, Hkv, record] uint8 of rows k, v [n, Hkv, d]."""
    n, H, d = np.shape(k)
    rec = np.zeros((n, H, kv4_record_bytes(d)), dtype=np.uint8)
    for half, x in enumerate((k, v)):
        byte, q = kv4_quantise(x)
        code = (q + 8).astype(np.uint32).reshape(n, H, d // 8, 8)
        word = np.zeros((n, H, d // 8), dtype=np.uint32)
        for e in range(8):
            word |= code[..., e] << np.uint32(4 * (e // 2) + 16 * (e % 2))
        rec[:, :, half * d // 2:(half + 1) * d // 2] = word.astype("<u4").view(np.uint8).reshape(n, H, d // 2)
        rec[:, :, d + half * d // 16:d + (half + 1) * d // 16] = byte
    return rec


def kv4_unpack(rec, d: int):
    """((scale bytes, multiples) of K, the same of V) from records."""
    rec = np.asarray(rec)
    out = []
    for half in (0, 1):
        word = np.ascontiguousarray(rec[..., half * d // 2:(half + 1) * d // 2]).view("<u4")
        q = np.stack([(word >> np.uint32(4 * (e // 2) + 16 * (e % 2))) & 15 for e in range(8)], axis=-1)
        out.append((rec[..., d + half * d // 16:d + (half + 1) * d // 16],
                    q.astype(np.int64).reshape(*rec.shape[:-1], d) - 8))
    return out


def kv4_values(rec, d: int):
    """(K, V) float64 values of records [..., record]."""
    return tuple(q * np.repeat(SCALES[byte], 16, axis=-1) for byte, q in kv4_unpack(rec, d))
