"""8-bit activation checkpoints on the host: the oracle's pins and the refusals
of the C ABI and the Python binding (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import segment_masked_causal_gb300 as pa
from oracle import checkpoint as ck

FAKE = 0x100000  # a 16-byte-aligned non-null address; never dereferenced on refusal


@pytest.fixture(scope="module")
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


def test_oracle_e4m3_values_are_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert (codes == ck.E4M3).all()
    # and rounding agrees with torch's on fp32 values, ties among them
    y = np.concatenate([(ck.E4M3[1:] + ck.E4M3[:-1]) / 2, np.random.default_rng(3).uniform(0, 448, 5000)]).astype(np.float32)
    assert (torch.tensor(y).to(torch.float8_e4m3fn).double().numpy() == ck.E4M3[ck.nearest_e4m3(y.astype(np.float64))]).all()


def test_oracle_hand_worked_block():
    x = np.zeros((1, 32))
    x[0, :5] = [127.0, -63.5, 0.5, 1.5, -126.4]
    v, s = ck.save(x, "int8", 32)
    assert s[0, 0] == 1.0 and (v[0, :5] == [127, -64, 0, 2, -126]).all()  # halves go to the even code
    x[0, :5] = [448.0, 17.0, -19.0, 2.0 ** -10, 3 * 2.0 ** -10]
    v, s = ck.save(x, "e4m3", 32)
    assert s[0, 0] == 1.0 and (v[0, :5] == [448, 16, -20, 0, 2.0 ** -8]).all()
    x[0, 7] = np.inf
    v, s = ck.save(x, "int8", 32)
    assert np.isnan(s[0, 0]) and (v == 0).all()
    v, s = ck.save(np.zeros((2, 40)), "int8", 32)
    assert (s == 0).all() and s.shape == (2, 2) and (v == 0).all()


def _t(B=1, H=2, N=3, C=64, sb=None, sh=None, sn=None, x=FAKE, c=FAKE, s=FAKE):
    sn = C if sn is None else sn
    sh = N * sn if sh is None else sh
    sb = H * sh if sb is None else sb
    return pa.pa_ckpt_tensor(x, c, s, B, H, N, C, sb, sh, sn)


@pytest.mark.parametrize("name", ["pa_ckpt_save", "pa_ckpt_load"])
def test_refusals(L, name):
    fn = getattr(L, name)

    def f(*ts, io=0, fmt=0, block=64, count=None):
        ts = ts or (_t(),)
        return fn(len(ts) if count is None else count, (pa.pa_ckpt_tensor * len(ts))(*ts), io, fmt, block, None)
    assert fn(1, None, 0, 0, 64, None) == 1
    assert f(count=0) == 4 and f(*[_t()] * 9) == 4
    assert f(block=16) == 4 and f(block=96) == 4 and f(io=2) == 9 and f(fmt=2) == 9 and f(fmt=-1) == 9
    for bad in (dict(B=0), dict(H=0), dict(N=0), dict(C=0), dict(C=60), dict(sn=56), dict(sh=8), dict(B=2, sb=0)):
        assert f(_t(**bad)) == 4, bad
    assert f(_t(sn=68)) == 5 and f(_t(sn=66), io=1) == 5
    assert f(_t(x=None)) == 1 and f(_t(c=None)) == 1 and f(_t(s=None)) == 1
    assert f(_t(x=FAKE + 8)) == 5 and f(_t(c=FAKE + 4)) == 5 and f(_t(s=FAKE + 8)) == 5
    assert f(_t(), _t(C=4)) == 4  # any tensor of the list
    # groups of eight elements are counted in 31 bits
    assert f(_t(B=1 << 20, H=1 << 10, N=1 << 10, C=8)) == 4
    assert f(_t(B=2, H=1, N=(1 << 30) - 100, C=16)) == 4
    assert f(_t(B=2147483647, H=2147483647, N=2147483647, C=8)) == 4
    if not torch.cuda.is_available():
        assert f() in (7, 8)
        # the stride of a dimension of one is never used
        assert f(_t(B=1, H=1, N=5, sb=3, sh=1)) in (7, 8)
        assert f(_t(sn=68), io=1) in (7, 8)


def test_backward_refusals(L):
    d = lambda B=1, Hq=4, Hkv=2, N=200, D=64: pa.make_dims(B, Hq, Hkv, N, D)
    need = L.pa_bwd_ckpt_workspace_bytes(ctypes.byref(d()))
    # the kernels' part for whole tiles, then q, k and v in bf16
    assert need >= L.pa_workspace_bytes(ctypes.byref(d(N=256))) + 200 * 64 * 2 * (4 + 2 + 2)
    assert L.pa_bwd_ckpt_workspace_bytes(None) == 0
    assert L.pa_bwd_ckpt_workspace_bytes(ctypes.byref(d(D=80))) == 0
    assert L.pa_bwd_ckpt_workspace_bytes(ctypes.byref(d(B=1 << 13, Hq=32, Hkv=32, N=8000, D=128))) == 0
    ok = pa.pa_ckpt(FAKE, FAKE)

    def f(dims=None, st=None, fmt=0, block=64, q=ok, out=ok, dout=FAKE, lse=FAKE, seg=FAKE, dq=FAKE, ws=FAKE, n=need):
        ref = lambda c: None if c is None else ctypes.byref(c)
        return L.pa_bwd_ckpt(ctypes.byref(dims or d()), None if st is None else ctypes.byref(st), fmt, block, ref(q),
                             ref(ok), ref(ok), ref(out), dout, lse, seg, dq, FAKE, FAKE, ws, n, None)
    assert f(d(D=80)) == 2 and f(d(Hq=3)) == 3 and f(d(N=0)) == 4
    assert f(block=48) == 4 and f(fmt=7) == 9
    assert f(q=None) == 1 and f(out=pa.pa_ckpt(FAKE, None)) == 1 and f(dout=None) == 1 and f(ws=None) == 1
    assert f(q=pa.pa_ckpt(FAKE + 8, FAKE)) == 5 and f(dq=FAKE + 8) == 5 and f(seg=FAKE + 4) == 5
    assert f(n=need - 1) == 6
    assert f(st=pa.pa_strides(1 << 20, 32, 256, 1 << 20, 64, 128)) == 4
    assert f(st=pa.pa_strides(1 << 20, 68, 256, 1 << 20, 64, 128)) == 5
    if not torch.cuda.is_available():
        assert f() in (7, 8) and f(seg=None) in (7, 8) and f(d(N=256), n=1 << 30) in (7, 8)


def test_python_refusals():
    c, s = torch.zeros(3, 64, dtype=torch.int8), torch.zeros(3, 1)
    pa.Checkpoint(c, s, 64)
    assert pa.Checkpoint(c, s, 64).nbytes == 3 * 64 + 12
    with pytest.raises(ValueError, match="scales"):
        pa.Checkpoint(c, s, 32)
    with pytest.raises(ValueError, match="block"):
        pa.Checkpoint(c, s, 16)
    with pytest.raises(ValueError, match="codes"):
        pa.Checkpoint(c.float(), s, 64)
    with pytest.raises(ValueError, match="format"):
        pa.checkpoint_save([c.bfloat16()], format="int4")
    with pytest.raises(ValueError, match="block"):
        pa.checkpoint_save([c.bfloat16()], block=50)
    assert pa.checkpoint_save([]) == [] and pa.checkpoint_load([]) == []


def test_a_dimension_past_31_bits_is_refused():
    """Tensors without storage: only their shapes matter. 1-D, and as one of four dims."""
    for shape in ((1 << 31,), (1, 1, (1 << 31) + 8, 8)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="meta")
        c = torch.empty(shape, dtype=torch.int8, device="meta")
        s = torch.empty((*shape[:-1], -(-shape[-1] // 64)), device="meta")
        with pytest.raises(pa.PAError, match="2\\^31"):
            pa._ckpt_of(x, c, s, x.get_device())
