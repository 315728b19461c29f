"""fp64 restatement of the 8-bit activation checkpoints (test infrastructure).

TEST INFRASTRUCTURE ONLY: only the tests may import this module; the library
never calls it and shares no code with it.

A row is cut into blocks; per block scale = fp32(max |x| / top), top = 127
(int8) or 448 (e4m3), and each element is kept as the value nearest to
x / scale among the format's values (ties to the even one), clamped to +-top.
e4m3's values are 0, the eight steps of 2^-9 below 2^-6, and (8 + i) / 8 * 2^k,
i < 8, k = -6..8, up to 448. The quotient of two fp32 values that is no tie
differs from it by more than fp64 loses, so fp64 decides every case.

Pins: tests/test_checkpoint_host.py (an enumeration of the e4m3 values, torch's
float8 type, hand-worked blocks).
"""
from __future__ import annotations

import numpy as np

TOP = {"int8": 127.0, "e4m3": 448.0}
E4M3 = np.array([i * 2.0 ** -9 for i in range(8)] +
                [(8 + i) / 8 * 2.0 ** k for k in range(-6, 9) for i in range(8)][:-1])  # the last code is NaN


def nearest_e4m3(y):
    """The index of the e4m3 magnitude nearest to |y| (ties to even)."""
    a = np.minimum(np.abs(y), 448.0)
    hi = np.searchsorted(E4M3, a).clip(1, len(E4M3) - 1)
    lo = hi - 1
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    return np.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), hi, lo)


def save(x, fmt, block):
    """(values, scales): what each element is kept as, in units of its scale
    (fp64), and the fp32 scales, blocks along the last axis."""
    x = np.asarray(x, np.float64)
    C, top = x.shape[-1], TOP[fmt]
    vals, scales = np.zeros_like(x), np.zeros(x.shape[:-1] + (-(-C // block),), np.float32)
    for j, a in enumerate(range(0, C, block)):
        b = x[..., a:a + block]
        ok = np.isfinite(b).all(axis=-1)
        m = np.where(ok, np.abs(np.where(np.isfinite(b), b, 0)).max(axis=-1), np.nan)
        s = (m / top).astype(np.float32)
        s64 = s.astype(np.float64)[..., None]
        with np.errstate(all="ignore"):
            y = np.where(s64 > 0, b / s64, 0.0)
        y = np.where(np.isnan(y), 0.0, y).clip(-top, top)
        vals[..., a:a + block] = np.rint(y) if fmt == "int8" else np.sign(y) * E4M3[nearest_e4m3(y)]
        scales[..., j] = s
    return vals, scales


def load(vals, scales, block):
    """The exact products code * scale."""
    C = vals.shape[-1]
    return vals * np.repeat(scales.astype(np.float64), block, axis=-1)[..., :C]
