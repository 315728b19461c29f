"""The checks of _paged_common.py against mistakes planted in the weights (no GPU needed):
they pass what rounding does and fail when one visit of a long context is lost, counted twice or weighted
by the wrong maximum."""
import numpy as np
import pytest
import torch

from _paged_common import RELATIVE, coded_values, relative, tolerance


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def case(n, D, seed, coded):
    rng = np.random.default_rng(seed)
    q, k = bf16(rng.normal(size=(4, D))), bf16(rng.normal(size=(n, D)))
    v = coded_values(n, 1, D)[:, 0].astype(np.float64) if coded else bf16(rng.normal(size=(n, D)))
    z = q @ k.T / np.sqrt(D)
    w = np.exp(z - z.max(1, keepdims=True))
    Z = (np.abs(q)[:, None] * np.abs(k)[None]).sum(-1).max(1) / np.sqrt(D)
    return w, v, Z


def finish(w, v):
    """As the kernel: rounded weights in the product, their exact sum below it."""
    return bf16(bf16(w) @ v / w.sum(1, keepdims=True))


def passes(got, w, v, Z, coded):
    p = w / w.sum(1, keepdims=True)
    want = p @ v
    if coded:
        return (np.abs(got - want) <= tolerance(want, p @ np.abs(v), Z)).all()
    return (relative(got, want) <= RELATIVE).all()


@pytest.mark.parametrize("coded", [False, True])
@pytest.mark.parametrize("n,D", [(20000, 64), (20000, 128), (12000, 96), (1100, 64)])
def test_rounding_passes_and_a_lost_visit_does_not(n, D, coded):
    for seed in range(3):
        w, v, Z = case(n, D, seed, coded)
        assert passes(finish(w, v), w, v, Z, coded)
        for at in (0, 128 * (n // 256), 128 * (n // 128 - 1)):
            for factor in (0.0, 2.0, np.exp(-2.0)):  # lost, twice, under another part's maximum
                u = w.copy()
                u[:, at:at + 128] *= factor
                bad = bf16(bf16(u) @ v / w.sum(1, keepdims=True))  # lse has the right sum
                assert not passes(bad, w, v, Z, coded), (seed, at, factor)
