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


@pytest.mark.parametrize("N", [32767, 32768, 32769, 33 * 1024 - 1, 33 * 1024, 33 * 1024 + 1, 1 << 20, 3_000_001])
@pytest.mark.parametrize("run", [1, 777, 1023, 1024, 1025, 4095, 4096, 5120, 5121, 6000, 70_000, 1 << 20, 1 << 31])
def test_runs_of_any_length(cuda_dev, N, run):
    """Around the length from which blocks leave marks, over runs that end inside, at and behind a block's border."""
    seg = runs(N, run, cuda_dev)
    if 4 * N < 1 << 22:  # more rows than one: what the one before leaves is not looked at
        seg = torch.cat([seg, seg.flip(1), seg + 1])
    got = pa.segment_positions(seg)
    for b in range(0, len(seg), 2):
        check(got[b], run)
    if len(seg) > 1:
        first = (N - 1) % run + 1  # the flipped row begins with the shorter run
        n = torch.arange(N, device=cuda_dev)
        assert torch.equal(got[1], torch.where(n < first, n, (n - first) % run).to(torch.int32))


def test_one_run_takes_time_in_proportion(cuda_dev):
    """A row of one run of 2^24 tokens: 16,384 blocks, each of which would look back over 8 million ids."""
    seg = torch.zeros(1, 1 << 24, dtype=torch.int32, device=cuda_dev)
    pos = torch.empty_like(seg)
    pa.pa_positions(seg, pos)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    pa.pa_positions(seg, pos)
    end.record()
    torch.cuda.synchronize()
    check(pos[0], 1 << 31)
    assert begin.elapsed_time(end) < 3  # 4,096 ids at a time it is 150 ms


def test_the_longest_row_of_one_run(cuda_dev):
    check(pa.segment_positions(torch.zeros(1, 2 ** 31 - 1, dtype=torch.int32, device=cuda_dev))[0], 1 << 31)
