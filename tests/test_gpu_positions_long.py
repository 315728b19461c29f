"""Positions of very long rows."""
import pytest
import torch

import segment_masked_causal_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


def check(got, run, chunk=1 << 26):
    """got (N): the positions of runs of `run` tokens each."""
    for a in range(0, len(got), chunk):
        n = torch.arange(a, min(a + chunk, len(got)), device=got.device)
        assert torch.equal(got[a:a + chunk], (n % run).to(torch.int32))


def runs(N, run, dev, chunk=1 << 26):
    seg = torch.empty(1, N, dtype=torch.int32, device=dev)
    for a in range(0, N, chunk):
        n = torch.arange(a, min(a + chunk, N), device=dev)
        seg[0, a:a + chunk] = (n // run).to(torch.int32)
    return seg


@pytest.mark.parametrize("N", [2 ** 31 - 1, 2 ** 31 - 1023, 2 ** 31 - 1024])
def test_the_longest_rows(cuda_dev, N):
    check(pa.segment_positions(runs(N, 1000, cuda_dev))[0], 1000)
