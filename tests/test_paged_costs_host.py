"""What a step of paged attention costs, by the kernel's own arithmetic on the host
(no GPU needed): the kernel adds the costs up in 32 bits, so their sum has to fit
for every step that the header allows, those of more tokens than the page table
lists or than kv_len counts among them."""
import ctypes

import numpy as np
import pytest

import segment_masked_causal_gb300 as pa


@pytest.fixture(scope="module")
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


def units(L, start, kv, Hq, Hkv, page, width, D=64):
    start, kv = np.asarray(start, np.int32), np.asarray(kv, np.int32)
    d = pa.pa_paged_dims(len(kv), int(start[-1]), Hq, Hkv, D, 1, page, width, 0.0)
    out = ctypes.c_uint64()
    assert L.pa_selftest_paged_units(ctypes.byref(d), start.ctypes.data, kv.ctypes.data, ctypes.byref(out)) == 0
    return out.value


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (32, 8), (128, 1), (64, 64), (8, 8)])
@pytest.mark.parametrize("page,width", [(16, 1), (64, 64), (256, (1 << 23) - 2)])
@pytest.mark.parametrize("T", [1, 200_000, 1 << 18, 1_200_000, 1 << 30])
def test_sum_fits_32_bits(L, Hq, Hkv, page, width, T):
    cap = page * width
    for S in (1, 2, 8, 3000):
        start = np.linspace(0, T, S + 1).astype(np.int64)
        for kv in (0, 1, min(T // S, 2 ** 31 - 1), cap, 2 ** 31 - 1, -5):
            n = units(L, start, np.full(S, kv), Hq, Hkv, page, width)
            assert (np.diff(start) > 0).sum() <= n < 1 << 32, (S, kv, n)


def test_uneven_sequences(L):
    # 200,000 new tokens of one sequence beside five of another, 4,096 keys in the table
    assert units(L, [0, 200_000, 200_005], [200_000, 5], 32, 8, 64, 64) < 1 << 32
    # as many sequences as a step may have, most of them without tokens
    S = (1 << 24) - 1
    start = np.zeros(S + 1, np.int32)
    start[S // 2:] = 1 << 20
    start[-1] = (1 << 20) + 1
    assert 2 <= units(L, start, np.full(S, 1 << 20, np.int32), 8, 1, 16, 4) < 1 << 32
    assert 1 << 24 <= units(L, np.arange(S + 2)[:S + 1] * 2, np.full(S, 7, np.int32), 1, 1, 16, 1) + 1 < 1 << 32


def test_hand_worked(L):
    # one token of 100 keys, table of 160: 100 - 1 keys and a fixed 320 and the token, for each of two kv heads
    assert units(L, [0, 1], [100], 2, 2, 16, 10) == 2 * (99 + 320 + 1)
    # a pair of tiles of 64 tokens each: 1.8 a key and 640
    assert units(L, [0, 128], [128], 2, 1, 16, 10) == int(np.float32(1.8) * np.float32(128) + np.float32(640))
    assert units(L, [0, 0], [100], 2, 2, 16, 10) == 0


def test_refusals(L):
    one = np.array([0, 1], np.int32)
    out = ctypes.c_uint64()

    def f(dims, a=one.ctypes.data, b=one.ctypes.data, o=ctypes.byref(out)):
        return L.pa_selftest_paged_units(dims, a, b, o)
    good = dict(S=1, T=1, Hq=2, Hkv=1, D=64, pages=1, page=16, width=1, scale=0.0)
    d = lambda **kw: ctypes.byref(pa.pa_paged_dims(*{**good, **kw}.values()))
    assert f(d()) == 0 and f(None) == 1 and f(d(), a=None) == 1 and f(d(), b=None) == 1 and f(d(), o=None) == 1
    assert f(d(D=80)) == 2 and f(d(Hq=129)) == 3 and f(d(S=0)) == 4 and f(d(page=8)) == 4


def test_no_size_is_refused_for_its_cost(L):
    """The most tokens over the longest table: what it costs fits (above), so the call goes ahead."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    fake = 0x100000
    d = pa.pa_paged_dims(1, 1 << 30, 4, 4, 64, 1, 256, (1 << 23) - 2, 0.0)
    s = pa.pa_paged_strides(256, 64, 0, 0, 256, 64, 65536, 16384, 64)
    n = L.pa_paged_workspace_bytes(64)
    assert L.pa_paged_fwd(ctypes.byref(d), ctypes.byref(s), *[fake] * 9, n, None) in (7, 8)
