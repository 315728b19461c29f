"""Rotary positions on the host: the oracle's pins, the frequencies and the
fixed-point turns of the C ABI, and its refusals (no GPU needed)."""
import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import segment_masked_causal_gb300 as pa
from oracle import rotary

FAKE = 0x100000  # a 16-byte-aligned non-null address; never dereferenced on refusal


@pytest.fixture(scope="module")
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


def test_oracle_hand_worked():
    # a quarter and a half turn, amplitude 2
    x = np.array([[1.0, 2.0, 3.0, 4.0, 9.0]])
    f = [math.pi / 2, math.pi]
    y = rotary.rotate(x, np.array([1]), f, 2.0)
    assert np.allclose(y, [[-6, -4, 2, -8, 9]])  # (1, 3) -> (-3, 1), (2, 4) -> (-2, -4)
    y = rotary.rotate(x, np.array([1]), f, 2.0, interleaved=True)
    assert np.allclose(y, [[-4, 2, -6, -8, 9]])
    assert (rotary.rotate(x, np.array([0]), f) == x).all()
    assert rotary.positions(np.array([[5, 5, 7, 7, 7, 5], [0, 1, 1, -2, -2, -2]])).tolist() == [
        [0, 1, 0, 1, 2, 0], [0, 0, 1, 0, 1, 2]]


def test_oracle_gradient_is_the_transpose():
    rng = np.random.default_rng(1)
    f = rotary.frequencies(8)
    x, g, pos = rng.normal(size=(5, 12)), rng.normal(size=(5, 12)), np.arange(5) * 37
    for inter in (False, True):
        y = rotary.rotate(x, pos, f, 1.3, inter)
        dx = rotary.rotate(g, pos, f, 1.3, inter, backward=True)
        assert np.isclose((y * g).sum(), (x * dx).sum())
        # and by differences
        e = np.zeros_like(x)
        e[2, 3] = 1e-6
        d = ((rotary.rotate(x + e, pos, f, 1.3, inter) - rotary.rotate(x - e, pos, f, 1.3, inter)) * g).sum() / 2e-6
        assert np.isclose(d, dx[2, 3])


def test_scores_depend_on_distance_only():
    rng = np.random.default_rng(2)
    f = rotary.frequencies(16)
    q, k = rng.normal(size=16), rng.normal(size=16)
    dot = lambda p, r: rotary.rotate(q, np.array(p), f) @ rotary.rotate(k, np.array(r), f)
    assert np.isclose(dot(7, 3), dot(1007, 1003)) and not np.isclose(dot(7, 3), dot(8, 3))


@pytest.mark.parametrize("rot", [8, 24, 64, 96, 128])
@pytest.mark.parametrize("kw", [{}, dict(theta=5e5), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                                dict(scaling="bands", factor=8.0, original=8192, low=1.0, high=4.0),
                                dict(scaling="bands", factor=2.0, original=2048)])
def test_frequencies(L, rot, kw):
    got, want = pa.Rotary(rot, **kw), rotary.frequencies(rot, **kw)
    assert np.allclose(got.frequencies, want, rtol=1e-14, atol=0)
    if kw.get("scaling") == "base":  # the ends of the range
        plain = rotary.frequencies(rot)
        assert want[0] == plain[0] and math.isclose(want[-1], plain[-1] / kw["factor"], rel_tol=1e-12)


def test_turns_are_the_frequencies_in_fixed_point(L):
    two_pi = Fraction("6.283185307179586476925286766559")
    given = [0.0, 1.0, 1e-3, 1e-9, 2 * math.pi, 7.5, -0.25, -1e-30]
    r = pa.Rotary(16, frequencies=given, interleaved=True, amplitude=1.5)
    assert r.c.rot == 16 and r.c.layout == 1 and r.c.amplitude == 1.5 and r.frequencies == tuple(given)
    for f, t in zip(given, r.c.turns):
        exact = Fraction(f) / two_pi
        off = (Fraction(t, 1 << 64) - exact) % 1
        # the quotient in a double and the fraction cut to 64 bits
        assert min(off, 1 - off) <= max(abs(exact), 1) * Fraction(1, 1 << 52)
    assert not any(r.c.turns[8:])


def test_init_refusals(L):
    f = (ctypes.c_double * 64)(*[1.0] * 64)
    c = pa.pa_rotary()
    init = lambda rot=16, layout=0, f=f, a=1.0, c=c: L.pa_rotary_init(None if c is None else ctypes.byref(c), rot, layout, f, a)
    assert init() == 0 and init(rot=128) == 0
    for rot in (0, -8, 4, 12, 136):
        assert init(rot=rot) == 4
    assert init(layout=2) == 9 and init(layout=-1) == 9
    assert init(f=None) == 1 and init(c=None) == 1
    for a in (math.nan, math.inf, 1e39):
        assert init(a=a) == 4
    assert init(f=(ctypes.c_double * 64)(math.nan)) == 4

    def freq(rot=16, scaling=0, theta=1e4, factor=2.0, original=1e3, low=1.0, high=4.0, out=f):
        return L.pa_rotary_frequencies(rot, scaling, theta, factor, original, low, high, out)
    assert all(freq(scaling=s) == 0 for s in range(4))
    assert freq(rot=10) == 4 and freq(scaling=4) == 9 and freq(theta=0.0) == 4 and freq(theta=math.inf) == 4 and freq(out=None) == 1
    assert freq(factor=0.0) == 0  # not looked at
    assert all(freq(scaling=s, factor=0.0) == 4 for s in (1, 2, 3))
    assert freq(scaling=3, original=0.0) == 4 and freq(scaling=3, low=4.0) == 4 and freq(scaling=3, high=math.nan) == 4
    with pytest.raises(ValueError, match="scaling"):
        pa.Rotary(16, scaling="cubic")
    with pytest.raises(ValueError, match="frequencies"):
        pa.Rotary(16, frequencies=[1.0] * 7)
    with pytest.raises(ValueError, match="no scaling"):
        pa.Rotary(16, frequencies=[1.0] * 8, scaling="linear", factor=2.0)
    with pytest.raises(pa.PAError):
        pa.Rotary(20)


def _t(H=3, N=5, D=64, x=FAKE, y=FAKE + (1 << 20), **kw):
    s = dict(x_b=H * N * D, x_h=N * D, x_n=D, y_b=H * N * D, y_h=N * D, y_n=D)
    s.update(kw)
    return pa.pa_rope_tensor(x, y, H, s["x_b"], s["x_h"], s["x_n"], s["y_b"], s["y_h"], s["y_n"])


def test_rope_refusals(L):
    r = pa.Rotary(64)

    def f(*ts, rotary=r.ref, count=None, B=2, N=5, D=64, io=0, pos=None):
        ts = ts or (_t(),)
        return L.pa_rope(rotary, len(ts) if count is None else count, (pa.pa_rope_tensor * len(ts))(*ts), B, N, D, io, pos, 0, None)
    assert f(rotary=None) == 1 and L.pa_rope(r.ref, 1, None, 1, 1, 64, 0, None, 0, None) == 1
    assert f(count=0) == 4 and f(*[_t()] * 5) == 4
    for kw in (dict(B=0), dict(N=0), dict(B=1 << 16, N=1 << 16), dict(D=56), dict(D=60), dict(D=264)):
        assert f(**kw) == 4, kw
    assert f(rotary=ctypes.byref(pa.pa_rotary())) == 4  # not initialised
    assert f(io=2) == 9 and f(pos=FAKE + 2) == 5
    for kw in (dict(H=0), dict(H=65536), dict(x_n=56), dict(y_h=8)):
        assert f(_t(**kw)) == 4, kw
    assert f(_t(x_n=68)) == 5 and f(_t(y_n=66), io=1) == 5
    assert f(_t(x=None)) == 1 and f(_t(y=None)) == 1 and f(_t(x=FAKE + 8)) == 5 and f(_t(y=FAKE + 8)) == 5
    assert f(_t(y=FAKE, y_n=128, y_h=640, y_b=1920)) == 4  # in place with other strides
    assert f(_t(), _t(H=0)) == 4
    if not torch.cuda.is_available():
        assert f() in (7, 8) and f(_t(y=FAKE)) in (7, 8) and f(_t(x_n=68), io=1) in (7, 8)
        assert f(_t(H=1, x_h=3, y_h=1, x_b=5 * 64, y_b=5 * 64)) in (7, 8)  # a dimension of one


def test_positions_refusals(L):
    f = lambda B=2, N=5, seg=FAKE, pos=FAKE: L.pa_positions(B, N, seg, pos, None)
    assert f(B=0) == 4 and f(N=-1) == 4 and f(B=1 << 16, N=1 << 15) == 4
    assert f(seg=None) == 1 and f(pos=None) == 1 and f(seg=FAKE + 4) == 5 and f(pos=FAKE + 8) == 5
    if not torch.cuda.is_available():
        assert f() in (7, 8)
