"""Paged attention where a step is larger than its tables: every row of every
sequence is written. Tolerances as in test_gpu_paged.py, whose derivation they share."""
import math

import numpy as np
import pytest
import torch

import segment_masked_causal_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


@pytest.mark.parametrize("lens,Hq,Hkv,keys", [
    ([1_200_000, 5], 1, 1, 16),        # one sequence whose costs alone pass 32 bits
    ([100_000, 100_000], 64, 8, 16),   # two whose sum does
    ([3, 200_000, 5], 32, 8, 4096),    # and one beside others, over a longer table
])
def test_more_tokens_than_the_table_lists(cuda_dev, lens, Hq, Hkv, keys):
    """Tokens past the table see the keys that it lists; so do those of a kv_len below the new tokens, from its
    start on. All rows against the same few keys, in blocks, in fp64."""
    D, page, S, T = 64, 16, len(lens), sum(lens)
    g = torch.Generator(device=cuda_dev).manual_seed(S)
    n = keys // page
    pool = torch.randn(2, S * n, Hkv, page, D, generator=g, device=cuda_dev).bfloat16()
    table = torch.arange(S * n, dtype=torch.int32, device=cuda_dev).view(S, n)
    start = [0] + np.cumsum(lens).tolist()
    kv = [m - (7 if i == 0 else 0) for i, m in enumerate(lens)]  # the first one's first seven tokens lie before its start
    kv[0] = max(kv[0], 1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda_dev)
    q = torch.randn(T, Hq, D, generator=g, device=cuda_dev, dtype=torch.bfloat16)
    cache = pa.PagedCache(pool[0], pool[1])
    out, lse = torch.full_like(q, 7.0), torch.full((T, Hq), 7.0, device=cuda_dev)
    ws = pa.paged_workspace(q, cache)
    pa.paged_forward(q, cache, table, i32(start), i32(kv), out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    scale, G = 1 / math.sqrt(D), Hq // Hkv
    for s in range(S):
        K, V = (x[s * n:(s + 1) * n].double().transpose(0, 1).reshape(Hkv, keys, D) for x in pool)
        # no row is left as it was, and blocks of them have the right values: the first, those at the table's
        # end, some in the middle and the last
        first, last = start[s], start[s + 1]
        assert not (lse[first:last] == 7).any() and not (out[first:last] == 7).all(-1).any()
        block = min(300, last - first)
        for a in sorted({min(first + x, last - block) for x in (0, max(0, keys - block // 2), (last - first) // 2, last - first)}):
            rows = torch.arange(a, a + block, device=cuda_dev)
            seen = (rows - first + kv[s] - lens[s] + 1).clamp(0, min(keys, kv[s]))
            z = torch.einsum("thgd,hkd->thgk", q[rows].double().view(-1, Hkv, G, D), K) * scale
            Z = torch.einsum("thgd,hkd->thgk", q[rows].double().abs().view(-1, Hkv, G, D), K.abs()).amax(-1).view(-1, Hq) * scale
            z = z.masked_fill(torch.arange(keys, device=cuda_dev) >= seen.view(-1, 1, 1, 1), -math.inf)
            wl = torch.logsumexp(z, -1)
            w = torch.exp(z - wl.clamp(min=-1e300)[..., None])
            want = torch.einsum("thgk,hkd->thgd", w, V).reshape(-1, Hq, D)
            A = torch.einsum("thgk,hkd->thgd", w, V.abs()).reshape(-1, Hq, D)
            wl = wl.view(-1, Hq)
            none = torch.isinf(wl)
            assert (none == (seen == 0).view(-1, 1)).all()
            assert (lse[rows][none] == -math.inf).all() and (out[rows][none] == 0).all()
            score = 10 * 2.0 ** -23 * Z
            tol = (2 * 2.0 ** -8 + 2.0 ** -12 + 2 * score[..., None]) * A + 2.0 ** -8 * want.abs()
            assert ((out[rows].double() - want).abs() <= tol).all()
            err = (lse[rows].double() - wl).abs()[~none]
            assert (err <= (score + 2.0 ** -22 + (64 + keys / 64) * 2.0 ** -24 + 2.0 ** -23 * wl.abs())[~none]).all()


@pytest.mark.parametrize("S,used", [(300, [0, 299]), (1000, [1, 33, 34, 162, 163, 900]), ((1 << 24) - 1, [0, 5_000_000, (1 << 24) - 2])])
def test_few_slots_in_use(cuda_dev, S, used):
    """A step of a program that keeps a slot for every sequence it may ever run: the slots without new
    tokens are passed in a fraction of the 2 s after which a kernel's waits give up."""
    D, page, width, kv_of = 64, 16, 4, [60, 3, 33, 64, 1, 17]
    n = len(used)
    g = torch.Generator(device=cuda_dev).manual_seed(S)
    pool = torch.randn(2, n * width, 2, page, D, generator=g, device=cuda_dev).bfloat16()
    cache = pa.PagedCache(pool[0], pool[1])
    at = torch.tensor(used, device=cuda_dev)
    own = torch.arange(n * width, device=cuda_dev, dtype=torch.int32).view(n, width)
    table = torch.full((S, width), -1, device=cuda_dev, dtype=torch.int32)
    kv, new = (torch.zeros(S, device=cuda_dev, dtype=torch.int32) for _ in range(2))
    lens = torch.tensor(kv_of[:n], device=cuda_dev, dtype=torch.int32)
    table[at], kv[at], new[at] = own, lens, 1
    start = torch.zeros(S + 1, device=cuda_dev, dtype=torch.int32)
    start[1:] = new.cumsum(0)
    q = torch.randn(n, 4, D, generator=g, device=cuda_dev, dtype=torch.bfloat16)
    want, wl = pa.paged_forward(q, cache, own, torch.arange(n + 1, device=cuda_dev, dtype=torch.int32), lens)  # the same slots alone
    out, lse, ws = torch.full_like(q, 7.0), torch.full((n, 4), 7.0, device=cuda_dev), pa.paged_workspace(q, cache)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    pa.paged_forward(q, cache, table, start, kv, out=out, lse=lse, ws=ws)
    end.record()
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    assert torch.equal(out, want) and torch.equal(lse, wl)  # contexts of one visit are never cut
    assert begin.elapsed_time(end) < 600


@pytest.mark.parametrize("S", [40, 8000])
def test_many_arrays_out_of_range_are_taken_into_it(cuda_dev, S):
    """q_start that rises and falls over many sequences, so that their rows add up to far more than T and
    their costs to more than 32 bits: nothing outside the tensors is touched, and the next step is as ever."""
    D, page, width, T = 64, 16, 2, 20_000
    rng = np.random.default_rng(S)
    guard = 64
    g = torch.Generator(device=cuda_dev).manual_seed(S)
    pool = torch.randn(2, 8, 1, page, D, generator=g, device=cuda_dev).bfloat16()
    cache = pa.PagedCache(pool[0], pool[1])
    i32 = lambda x: torch.from_numpy(np.asarray(x).astype(np.int32)).to(cuda_dev)
    table = i32(rng.integers(0, 8, (S, width)))
    q = torch.randn(T, 1, D, generator=g, device=cuda_dev).bfloat16()
    around = torch.full((T + 2 * guard, 1, D), 7.0, device=cuda_dev, dtype=torch.bfloat16)
    lse_all = torch.full((T + 2 * guard, 1), 7.0, device=cuda_dev)
    ws = pa.paged_workspace(q, cache)

    def step(start, kv, tab):
        pa.paged_forward(q, cache, tab, i32(start), i32(kv), out=around[guard:-guard], lse=lse_all[guard:-guard], ws=ws)
        torch.cuda.synchronize()
        assert pa.pa_device_status(ws) == 0
        assert (around[:guard] == 7).all() and (around[-guard:] == 7).all()
        assert (lse_all[:guard] == 7).all() and (lse_all[-guard:] == 7).all()
        return around[guard:-guard].clone(), lse_all[guard:-guard].clone()
    good = np.linspace(0, T, S + 1), np.full(S, 30)
    want = step(*good, table)
    step(np.tile([0, T], S // 2 + 1)[:S + 1], np.full(S, 30), table)
    bad = rng.integers(-2 ** 31, 2 ** 31, S + 1)
    step(bad, rng.integers(-2 ** 31, 2 ** 31, S), i32(rng.integers(-2 ** 31, 2 ** 31, (S, width))))
    assert all(torch.equal(x, y) for x, y in zip(want, step(*good, table)))
