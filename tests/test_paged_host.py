"""The paged cache on the host: the oracle's pins and the refusals of the C ABI
and the Python binding (no GPU needed)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import segment_masked_causal_gb300 as pa
from oracle import paged

FAKE = 0x100000  # a 16-byte-aligned non-null address; never dereferenced on refusal


@pytest.fixture(scope="module")
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


def test_oracle_hand_worked():
    # page 16, three tokens on page 2; two of them new; keys all zero, so weights are equal
    k, v = np.zeros((3, 1, 16, 4)), np.full((3, 1, 16, 4), np.nan)
    v[2, 0, :3] = [[1] * 4, [2] * 4, [6] * 4]
    q = np.ones((3, 2, 4))
    out, lse, A, Z = paged.attention(q, k, v, np.array([[2]]), [0, 2], [3])
    assert np.allclose(out[0], 1.5) and np.allclose(out[1], 3) and np.isnan(out[2]).all()
    assert np.allclose(lse[:2], [[math.log(2)] * 2, [math.log(3)] * 2])
    # a page that is not there, and a row that sees nothing
    out, lse, _, _ = paged.attention(q, k, v, np.array([[-1]]), [0, 2], [3])
    assert (out[:2] == 0).all() and (lse[:2] == -np.inf).all()
    out, lse, _, _ = paged.attention(q, k, v, np.array([[2]]), [0, 2], [1])
    assert (out[0] == 0).all() and np.allclose(out[1], 1)
    assert paged.places([0, 0, 3], [7, 17], np.array([[1, 2], [0, 5]]), 4, 16) == [
        (0, 1, 14, 0, 14), (1, 1, 15, 0, 15), (2, 1, 16, -1, 0)]


def test_oracle_is_the_packed_attention():
    rng = np.random.default_rng(4)
    Hq, Hkv, N, D, page = 4, 2, 40, 8, 16
    q, k, v = (rng.normal(size=(1, H, N, D)) for H in (Hq, Hkv, Hkv))
    ref = oracle.attention(q, k, v, np.zeros((1, N), np.int32), 1 / math.sqrt(D), q)
    kp, vp = np.zeros((4, Hkv, page, D)), np.zeros((4, Hkv, page, D))
    table = np.array([[3, 0, 2]])
    for j in range(N):
        kp[table[0, j // page], :, j % page], vp[table[0, j // page], :, j % page] = k[0, :, j], v[0, :, j]
    # the last 25 tokens as a chunk
    out, lse, _, _ = paged.attention(q[0].transpose(1, 0, 2)[-25:], kp, vp, table, [0, 25], [N])
    assert np.allclose(out, ref["o"][0].transpose(1, 0, 2)[-25:]) and np.allclose(lse, ref["lse"][0].T[-25:])


def dims(S=3, T=7, Hq=8, Hkv=2, D=64, pages=9, page=16, width=4, scale=0.0):
    return pa.pa_paged_dims(S, T, Hq, Hkv, D, pages, page, width, scale)


def strides(**kw):
    s = dict(q_t=512, q_h=64, n_t=128, n_h=64, o_t=512, o_h=64, p_p=2048, p_h=1024, p_n=64)
    s.update(kw)
    return pa.pa_paged_strides(*s.values())


BAD_SHAPES = [dict(S=0), dict(S=1 << 24), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(pages=0), dict(width=0), dict(page=8),
              dict(page=48), dict(page=512), dict(page=0), dict(width=1 << 27), dict(scale=math.inf), dict(Hq=65538), dict(T=(1 << 30) + 1)]


@pytest.mark.parametrize("call", ["append", "fwd"])
def test_refusals(L, call):
    r = pa.Rotary(64)
    need = L.pa_paged_workspace_bytes(64)

    def f(d=None, s=None, q=FAKE, k=FAKE, v=FAKE, table=FAKE, start=FAKE, kv=FAKE, out=FAKE, kp=FAKE, vp=FAKE, rotary=r.ref,
          pos=None, lse=FAKE, ws=FAKE, n=need):
        d, s = ctypes.byref(d or dims()), ctypes.byref(s or strides())
        if call == "append":
            return L.pa_paged_append(d, s, rotary, q, k, v, table, start, kv, pos, out, kp, vp, None)
        return L.pa_paged_fwd(d, s, q, kp, vp, table, start, kv, out, lse, ws, n, None)
    for kw in BAD_SHAPES:
        assert f(dims(**kw)) == 4, kw
    assert f(dims(D=80)) == 2 and f(dims(Hq=7)) == 3
    for name in ("q_t", "q_h", "o_t", "o_h", "p_p", "p_h", "p_n") + (("n_t", "n_h") if call == "append" else ()):
        assert f(s=strides(**{name: 56})) == 4 and f(s=strides(**{name: 1 << 38})) == 4 and f(s=strides(**{name: 4100})) == 5, name
    for name in ("table", "start", "kv", "kp", "vp") + (("k", "v") if call == "append" else ("q", "out", "lse", "ws")):
        assert f(**{name: None}) == 1, name
    for name in ("q", "out", "kp", "vp") + (("k", "v") if call == "append" else ("lse", "ws")):
        assert f(**{name: FAKE + 8}) == 5, name
    for name in ("table", "start", "kv") + (("pos",) if call == "append" else ()):
        assert f(**{name: FAKE + 2}) == 5, name
    if call == "append":
        assert f(q=None) == 1 and f(out=None) == 1  # they come together
        assert f(rotary=ctypes.byref(pa.pa_rotary())) == 4 and f(rotary=pa.Rotary(96).ref) == 4
        assert f(s=strides(o_t=1024)) == 4  # in place with other strides
    else:
        assert f(dims(Hq=258)) == 3 and f(n=need - 1) == 6
        assert L.pa_paged_workspace_bytes(80) == 0 and L.pa_paged_workspace_bytes(128) > 0
    assert f(dims(T=0), q=None, out=None, k=None, lse=None) == 0  # nothing to do
    if not torch.cuda.is_available():
        assert f() in (7, 8) and f(table=FAKE + 4) in (7, 8)
        assert f(dims(T=1, Hq=1, Hkv=1, pages=1), strides(q_t=1, q_h=3, n_t=5, n_h=7, o_t=9, o_h=11, p_p=2, p_h=4),
                 out=FAKE + 16) in (7, 8)


def test_python_refusals():
    k = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    pa.PagedCache(k, k.clone())
    assert pa.PagedCache(k, k).page == 16
    with pytest.raises(ValueError, match="pages"):
        pa.PagedCache(k, k[:2])
    with pytest.raises(ValueError, match="bfloat16"):
        pa.PagedCache(k.float(), k.float())
    with pytest.raises(ValueError, match="strides"):
        pa.PagedCache(k, k.transpose(1, 2).contiguous().transpose(1, 2))
    with pytest.raises(ValueError, match="contiguous"):
        pa.PagedCache(k.transpose(2, 3), k.transpose(2, 3))
