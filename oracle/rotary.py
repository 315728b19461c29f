"""Rotary positions in fp64, from the definition: pairs as complex numbers
turned by position times frequency."""
import math

import numpy as np


def frequencies(rot, theta=10000.0, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    if scaling == "base":
        theta = theta * factor ** (rot / (rot - 2))
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        out = []
        for x in f:
            turns = original * x / (2 * math.pi)
            keep = min(1.0, max(0.0, (turns - low) / (high - low)))
            out.append(keep * x + (1 - keep) * x / factor)
        return np.array(out)
    return f


def positions(seg):
    out = np.zeros(seg.shape, np.int32)
    for b in range(seg.shape[0]):
        for n in range(1, seg.shape[1]):
            out[b, n] = out[b, n - 1] + 1 if seg[b, n] == seg[b, n - 1] else 0
    return out


def members(rot, interleaved):
    """Indexes of the first and second elements of the pairs."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, pos, freq, amplitude=1.0, interleaved=False, backward=False):
    """x (..., D) fp64 with pos (...,) broadcast against its leading dims."""
    a, b = members(2 * len(freq), interleaved)
    # the angle in long double (64 bits or more), without its whole turns before it is a double again
    angle = np.asarray(pos, np.longdouble)[..., None] * np.asarray(freq, np.longdouble)
    angle = np.asarray(np.fmod(angle, 8 * np.arctan(np.longdouble(1))), np.float64)
    z = (x[..., a] + 1j * x[..., b]) * amplitude * np.exp((-1j if backward else 1j) * angle)
    y = x.copy()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def weight(x, freq, interleaved=False):
    """|x1| + |x2| of each element's pair (0 where an element has none): what its rounding errors scale with."""
    a, b = members(2 * len(freq), interleaved)
    w = np.zeros_like(x)
    w[..., a] = w[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return w
