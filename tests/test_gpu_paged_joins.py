"""Long contexts cut into parts and joined, to the bars of _paged_common.py, which tell a
lost or misweighted visit of 128 keys from rounding."""
import numpy as np
import pytest
import torch

from _paged_common import RELATIVE, coded_values, relative, tolerance
from oracle import paged
from test_gpu_paged import Step, built, f64  # noqa: F401

pytestmark = pytest.mark.gpu


def code(s):
    """Coded values in the places of the sequences' own."""
    for i, (_, t) in enumerate(s.lens):
        v = torch.from_numpy(coded_values(t, s.vp.shape[1], s.D)).to(s.dev, s.vp.dtype)
        for j in range(0, t, s.page):
            n = min(s.page, t - j)
            s.vp[int(s.table[i, j // s.page]), :, :n] = v[j:j + n].transpose(0, 1)


def check(s, coded):
    out, lse = s.forward()
    want, wl, A, Z = paged.attention(f64(s.q), f64(s.kp), f64(s.vp), s.table, s.start, s.kv)
    got = f64(out)
    assert (np.abs(got - want) <= tolerance(want, A, Z)).all()
    bar = 10 * 2.0 ** -23 * Z + 2.0 ** -22 + (64 + max(t for _, t in s.lens) / 64) * 2.0 ** -24 + 2.0 ** -23 * np.abs(wl)
    assert (np.abs(f64(lse) - wl) <= bar).all()
    if not coded:
        assert (relative(got, want) <= RELATIVE).all(), relative(got, want).max()


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("lens", [[(1, 20000)], [(2, 12000)], [(9, 12009)], [(40, 12040)], [(100, 12100)],
                                  [(3, 9000), (1, 50), (100, 5000), (1, 1100)], [(1, 700 * i + 5) for i in range(1, 25)]],
                         ids=["one", "two", "few", "tile", "pair", "mixed", "many"])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (5, 1, 96), (8, 2, 128)])
def test_parts_are_joined(cuda_dev, lens, Hq, Hkv, D, coded):
    s = Step(lens, Hq, Hkv, D, 64, cuda_dev, seed=D + len(lens))
    if coded:
        code(s)
    check(s, coded)


@pytest.mark.parametrize("D,Hq,page", [(64, 2, 16), (128, 16, 256)])
def test_parts_of_very_different_weight(cuda_dev, D, Hq, page):
    """Scores that rise along the context, so that each part's maximum is another and the last parts hold most of
    the weight; and ones that fall."""
    for sign in (1, -1):
        s = Step([(1, 9000), (5, 6000)], Hq, 1, D, page, cuda_dev, seed=D)
        for i, (_, t) in enumerate(s.lens):
            for j in range(0, t, page):
                n = min(page, t - j)
                s.kp[int(s.table[i, j // page]), :, :n, 0] = sign * (j / t) * 8
        s.q[:, :, 0] = 8.0
        code(s)
        check(s, True)
