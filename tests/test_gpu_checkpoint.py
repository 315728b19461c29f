"""8-bit activation checkpoints on the GPU, and the attention backward from
them, against the fp64 oracles.

Save and load are exact operations with one rounding each, so their results
have to be the oracle's to the bit: scales, the kept values, and the loaded
values (code * scale rounded to fp32, then to the tensor's type)."""
import math

import numpy as np
import pytest
import torch

import oracle
import segment_masked_causal_gb300 as pa
import synth
from oracle import checkpoint as ck

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


def values(codes):
    return codes.float().cpu().numpy().astype(np.float64)


def check(x, c, y):
    """Checkpoint c of x and its load y, all on the device."""
    fmt = "int8" if c.codes.dtype == torch.int8 else "e4m3"
    with np.errstate(over="ignore"):
        v, s = ck.save(x.float().cpu().numpy(), fmt, c.block)
    got = c.scales.cpu().numpy()
    assert got.dtype == np.float32 and np.array_equal(got, s, equal_nan=True)
    assert np.array_equal(values(c.codes), v)
    rep = np.repeat(s, c.block, axis=-1)[..., :x.shape[-1]]
    with np.errstate(over="ignore"):  # the largest finite value times 448 / 448 rounded up
        want = torch.from_numpy(v.astype(np.float32) * rep).to(x.dtype)
    assert y.dtype == x.dtype and y.shape == x.shape
    assert np.array_equal(y.float().cpu().numpy(), want.float().numpy(), equal_nan=True)


def roundtrip(x, fmt, block):
    c = pa.checkpoint_save([x], format=fmt, block=block)[0]
    y = pa.checkpoint_load([c])[0]
    torch.cuda.synchronize()
    check(x, c, y)
    return c, y


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("block", [32, 64, 128])
@pytest.mark.parametrize("shape", [(8,), (1, 8), (3, 64), (5, 200), (2, 3, 7, 96), (1, 4, 130, 128), (1000, 72), (3, 4104)])
def test_save_and_load_are_exact(shape, block, dtype, fmt, cuda_dev):
    g = torch.Generator(device=cuda_dev).manual_seed(len(shape) * 1000 + shape[-1])
    x = (torch.randn(shape, generator=g, device=cuda_dev) * 3).to(dtype)
    roundtrip(x, fmt, block)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_ties_and_neighbours_of_ties(fmt, dtype, cuda_dev):
    """Blocks whose scale is a power of two, with every border between two
    codes and the fp32 values on either side of it."""
    top = ck.TOP[fmt]
    mids = np.arange(-126.5, 127) if fmt == "int8" else np.concatenate([[-1, 1] * ((ck.E4M3[1:] + ck.E4M3[:-1]) / 2)[:, None]])
    mids = np.asarray(mids, np.float32).reshape(-1)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(1e9)), np.nextafter(mids, np.float32(-1e9))])
    near = np.concatenate([near, np.zeros(-len(near) % 31, np.float32)]).reshape(-1, 31)
    x = np.concatenate([np.full((len(near), 1), top, np.float32), near], 1)
    for e in (0, -20, 30, -126, -140):
        roundtrip(torch.from_numpy(np.ldexp(x, e).astype(np.float32)).to(cuda_dev).to(dtype), fmt, 32)
    # scales of full width: many quotients, some within a rounding of a border
    u = synth.normals(3, 70, 64 * 4096).reshape(4096, 64).astype(np.float32)
    roundtrip(torch.from_numpy(u).to(cuda_dev).to(dtype), fmt, 64)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_fp32_quotients_that_meet_a_border(fmt, cuda_dev):
    """x = fp32(border * scale) for random scales: the quotient lies within
    half a step of fp32 of the border, on either side or on it."""
    top = np.float32(ck.TOP[fmt])
    u = np.abs(synth.normals(5, 71, 3000)).astype(np.float32) + np.float32(0.01)
    amax = u * top
    s = (amax.astype(np.float64) / float(top)).astype(np.float32)
    mids = (np.arange(0.5, 127) if fmt == "int8" else (ck.E4M3[1:] + ck.E4M3[:-1]) / 2).astype(np.float64)
    pick = (synth.uint64s(5, 72, 3000 * 31) % np.uint64(len(mids))).astype(np.int64).reshape(3000, 31)
    x = (mids[pick] * s[:, None].astype(np.float64)).astype(np.float32)
    x *= np.where(synth.uint64s(5, 73, x.size).reshape(x.shape) % np.uint64(2) == 0, np.float32(1), np.float32(-1))
    roundtrip(torch.from_numpy(np.concatenate([amax[:, None], x], 1)).to(cuda_dev), fmt, 32)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_tiny_huge_and_broken_blocks(fmt, dtype, cuda_dev):
    x = torch.randn(12, 64, device=cuda_dev, generator=torch.Generator(device=cuda_dev).manual_seed(1))
    x[0] = 0
    x[1] *= 1e-38
    x[2] *= 2e-44  # subnormal in fp32: scales of a bit or two
    x[3] = 0
    x[3, 5] = 1.4e-45 if dtype == torch.float32 else 1e-40
    x[4] *= 1e37
    x[5, 3] = float("inf")
    x[6, 33] = float("nan")
    x[7, 40] = -float("inf")
    x[8] = -0.0
    x[9] = torch.finfo(dtype).max
    x[10, :32] = 0
    x[11] = 1e-30 * x[11]
    x = x.to(dtype)
    c, y = roundtrip(x, fmt, 32)
    assert torch.isnan(y[5, :32]).all() and torch.isfinite(y[5, 32:]).all()
    assert torch.isfinite(y[6, :32]).all() and torch.isnan(y[6, 32:]).all() and torch.isnan(y[7, 32:]).all()
    assert (y[0] == 0).all() and (y[10, :32] == 0).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_strided_tensors_many_at_once_and_nothing_else_touched(fmt, cuda_dev):
    """(B, N, H, D) memory, rows with gaps and slices, eleven tensors (two
    launches); what lies between the rows of a destination stays."""
    g = torch.Generator(device=cuda_dev).manual_seed(2)
    mem = torch.randn(2, 33, 5, 96, generator=g, device=cuda_dev).bfloat16()
    wide = torch.randn(50, 256, generator=g, device=cuda_dev).bfloat16()
    xs = [mem.transpose(1, 2), mem.transpose(1, 2)[:, 1:4], mem[:, :, 2], wide[:, 64:136], wide[::2, 8:72], wide[3:4],
          mem[1], wide[7], mem.transpose(1, 2)[:, :, 5:6], wide[:, :8], mem[:1, :1, :1]]
    kept = pa.checkpoint_save(xs, format=fmt, block=64)
    ys = pa.checkpoint_load(kept)
    torch.cuda.synchronize()
    for x, c, y in zip(xs, kept, ys):
        check(x, c, y)
    dst = torch.full((50, 256), 7.0, device=cuda_dev, dtype=torch.bfloat16)
    pa.checkpoint_load([kept[3], kept[4]], out=[dst[:, 64:136], dst[::2, 192:256]])
    torch.cuda.synchronize()
    assert torch.equal(dst[:, 64:136], ys[3]) and torch.equal(dst[::2, 192:256], ys[4])
    dst[:, 64:136] = 7
    dst[::2, 192:256] = 7
    assert (dst == 7).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("block", [32, 64, 128])
def test_fp32_strides_and_alignments(block, fmt, cuda_dev):
    """Every form of the fp32 kernels' accesses: whole tensors of whole blocks,
    rows on 32 bytes with gaps or short blocks, rows on 16 bytes only (a start
    16 bytes past a 32-byte boundary, a row stride of 4 mod 8 elements)."""
    g = torch.Generator(device=cuda_dev).manual_seed(4)
    mem = torch.randn(2, 37, 5, 96, generator=g, device=cuda_dev)
    wide = torch.randn(60, 268, generator=g, device=cuda_dev)  # 4 mod 8 elements a row
    flat = torch.randn(60 * 136 + 4, generator=g, device=cuda_dev)
    off = flat[4:].view(60, 136)
    for xs in ([mem.transpose(1, 2), mem.transpose(1, 2)[:, 1:4], mem[:, :, 2], mem[1]],  # 32-byte rows
               [off], [off[:, :128]], [wide[:, :128]], [wide[:, 4:140], wide[::3, 8:264], wide[7:8, :8], mem[0]],
               [flat[4:132]], [torch.randn(33, 256, generator=g, device=cuda_dev)]):
        assert all(x.data_ptr() % 16 == 0 for x in xs)
        kept = pa.checkpoint_save(xs, format=fmt, block=block)
        ys = pa.checkpoint_load(kept)
        torch.cuda.synchronize()
        for x, c, y in zip(xs, kept, ys):
            check(x, c, y)
    # into rows on 16 bytes, whose neighbours stay
    dst = torch.full((60, 268), 7.0, device=cuda_dev)
    kept = pa.checkpoint_save([wide[:, 4:140]], format=fmt, block=block)
    pa.checkpoint_load(kept, out=[dst[:, 4:140]])
    torch.cuda.synchronize()
    check(wide[:, 4:140], kept[0], dst[:, 4:140])
    assert (dst[:, :4] == 7).all() and (dst[:, 140:] == 7).all()


@pytest.mark.parametrize("C", [4096, 4104])  # whole blocks, and a short one in each row
def test_offsets_past_32_bits(C, cuda_dev):
    """More than 2^32 bytes and 2^31 elements: the last rows are kept like any."""
    N = (1 << 31) // C + 700
    x = torch.empty(N, C, dtype=torch.bfloat16, device=cuda_dev)
    x[:-1000] = 1
    tail = torch.randn(1000, C, generator=torch.Generator(device=cuda_dev).manual_seed(3), device=cuda_dev).bfloat16()
    x[-1000:] = tail
    c, = pa.checkpoint_save([x], block=64)
    y, = pa.checkpoint_load([c])
    torch.cuda.synchronize()
    check(tail, pa.Checkpoint(c.codes[-1000:], c.scales[-1000:], 64), y[-1000:])
    assert (c.codes[:-1000].amin() == 127).item() and (y[:-1000].amin() == y[:-1000].amax()).item()


def test_capture_and_streams(cuda_dev):
    x = torch.randn(300, 512, device=cuda_dev).bfloat16()
    want, = pa.checkpoint_load(pa.checkpoint_save([x]))
    graph = torch.cuda.CUDAGraph()
    static = torch.zeros_like(x)
    with torch.cuda.graph(graph):
        got, = pa.checkpoint_load(pa.checkpoint_save([static]))
    static.copy_(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again, = pa.checkpoint_load(pa.checkpoint_save([x]))
    side.synchronize()
    assert torch.equal(again, want)


def test_refusals(cuda_dev):
    x = torch.zeros(4, 64, device=cuda_dev, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        pa.checkpoint_save([x, x.float()])
    with pytest.raises(ValueError):
        pa.checkpoint_save([x.half()])
    with pytest.raises(ValueError):
        pa.checkpoint_save([x.t()])
    with pytest.raises(ValueError):
        pa.checkpoint_save([x.cpu()])
    with pytest.raises(pa.PAError):
        pa.checkpoint_save([x[:, :12]])
    with pytest.raises(pa.PAError):
        pa.checkpoint_save([x[:, 4:12]])  # starts 8 bytes into a row
    with pytest.raises(pa.PAError):
        pa.checkpoint_save([x[:0]])
    c = pa.checkpoint_save([x])[0]
    with pytest.raises(ValueError):
        pa.checkpoint_load([c], out=[x[:2]])


# ------------------------------------------------------- attention backward
# P and dS enter the products in bf16 and the gradients are stored in bf16, each
# off by at most 2^-8 of the value: with random signs about 2.3e-3 of the
# norm; the bar is the one of the attention gradients' tests.
GRAD_RELL2 = 2e-2

CASES = [
    # B, Hq, Hkv, N, D, segments, format, block, memory order
    (1, 2, 2, 1, 64, False, "int8", 64, "bhnd"),
    (1, 2, 1, 128, 64, True, "int8", 32, "bhnd"),
    (2, 4, 2, 200, 96, True, "e4m3", 32, "bnhd"),
    (1, 4, 1, 384, 128, True, "int8", 128, "bhnd"),
    (2, 2, 2, 256, 96, False, "int8", 64, "bnhd"),
    (1, 8, 2, 333, 64, True, "e4m3", 128, "bhnd"),
    (1, 2, 2, 511, 128, False, "e4m3", 64, "bnhd"),
]


def _rows(seed, stream, B, H, N, D, order, dev):
    b = torch.from_numpy(synth.bf16_normal(seed, stream, (B, N, H, D) if order == "bnhd" else (B, H, N, D)).view(np.int16))
    b = b.view(torch.bfloat16).to(dev)
    return b.transpose(1, 2) if order == "bnhd" else b


def _case(B, Hq, Hkv, N, D, segs, fmt, block, order, dev):
    q, k, v, do = (_rows(N + D, 80 + i, B, H, N, D, order, dev) for i, H in enumerate((Hq, Hkv, Hkv, Hq)))
    seg = None
    if segs:
        ids = np.stack([synth.lengths_to_ids(synth.uniform_lengths(N + b, N, 1, 60)) for b in range(B)]).astype(np.int32)
        seg = torch.from_numpy(ids).to(dev)
    out, lse = pa.forward(q, k, v, seg)
    kept = pa.checkpoint_save([q, k, v, out], format=fmt, block=block)
    return q, k, v, do, seg, out, lse, kept


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def _oracle(kept, do, lse, seg, D):
    loaded = [c.codes.float() * c.scales.repeat_interleave(c.block, -1)[..., :D] for c in kept]
    q, k, v = (f64(x.bfloat16()) for x in loaded[:3])
    o, g = f64(loaded[3]), f64(do)
    delta, l64 = (o * g).sum(-1), lse.double().cpu().numpy()
    s = None if seg is None else seg.cpu().numpy()
    scale = 1 / math.sqrt(D)
    dk, dv = oracle.dkv(q, k, v, s, scale, g, l64, delta)
    return oracle.dq(q, k, v, s, scale, g, l64, delta), dk, dv


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_backward_from_checkpoint_matches_oracle(case, cuda_dev):
    B, Hq, Hkv, N, D = case[:5]
    q, k, v, do, seg, out, lse, kept = _case(*case, cuda_dev)
    ws = torch.empty(pa.pa_bwd_ckpt_workspace_bytes(B, Hq, Hkv, N, D), dtype=torch.uint8, device=cuda_dev)
    got = pa.backward_from_checkpoint(*kept, do, lse, seg, ws=ws)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    for x, y, n in zip(got, _oracle(kept, do, lse, seg, D), ("dq", "dk", "dv")):
        norm = np.linalg.norm(y)
        rel = np.linalg.norm(f64(x) - y) / norm if norm > 1e-6 else np.abs(f64(x)).max()
        print(f"{n}: relL2 {rel:.2e}")
        assert rel <= GRAD_RELL2, n
    assert got[0].stride() == do.stride()
    again = pa.backward_from_checkpoint(*kept, do, lse, seg)
    for x, y in zip(got, again):
        assert torch.equal(x, y)


# Rounding normals to bf16 costs 1.66e-3 of their norm (the mean of a uniform error
# of half a step, 2^-8 of the power of two below). dv takes P and itself, dq and dk
# dS and themselves, in bf16: two roundings, 2.35e-3. What else there is, fp32 sums
# and exponentials, is below 1e-5. P rounded before it enters dS would make it
# three, 2.87e-3, and an error of delta of 1% where dout is about out (delta is then
# as large as any <dO, v>) much more. So 2.6e-3 is the bar; for a sample's spread,
# over 10^4 elements and more, 1% of that.
TWO_ROUNDINGS = 2.6e-3

LONG = [
    (1, 4, 1, 1500, 128, (100, 900), "int8", 64, "bhnd"), (2, 4, 2, 1000, 96, (64, 300), "e4m3", 32, "bnhd"),
    (1, 2, 2, 1301, 64, None, "int8", 128, "bnhd"), (1, 6, 2, 1024, 128, None, "e4m3", 128, "bhnd"),
    (3, 2, 1, 640, 64, (1, 60), "int8", 32, "bhnd"),
]


@pytest.mark.parametrize("case", LONG, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("like_out", [False, True])
def test_gradients_from_checkpoints_are_two_roundings_off(case, like_out, cuda_dev):
    B, Hq, Hkv, N, D, lens, fmt, block, order = case
    q, k, v, do = (_rows(N + D, 80 + i, B, H, N, D, order, cuda_dev) for i, H in enumerate((Hq, Hkv, Hkv, Hq)))
    seg = None
    if lens:
        ids = np.stack([synth.lengths_to_ids(synth.uniform_lengths(N + b, N, *lens)) for b in range(B)]).astype(np.int32)
        seg = torch.from_numpy(ids).to(cuda_dev)
    out, lse = pa.forward(q, k, v, seg)
    if like_out:
        do = (out.float() + 0.1 * do.float()).bfloat16()
    kept = pa.checkpoint_save([q, k, v, out], format=fmt, block=block)
    got = pa.backward_from_checkpoint(*kept, do, lse, seg)
    torch.cuda.synchronize()
    for x, y, n in zip(got, _oracle(kept, do, lse, seg, D), ("dq", "dk", "dv")):
        rel = np.linalg.norm(f64(x) - y) / np.linalg.norm(y)
        print(f"{n}: relL2 {rel:.2e}")
        assert rel <= TWO_ROUNDINGS, n


@pytest.mark.parametrize("D", [64, 96, 128])
def test_backward_with_rows_on_16_bytes(D, cuda_dev):
    """dout and its gradient with a row stride of 8 mod 16 elements and a start 16
    bytes past a 32-byte boundary; then a workspace that starts so, too."""
    B, Hq, Hkv, N = 2, 4, 2, 300
    q, k, v, do, seg, out, lse, kept = _case(B, Hq, Hkv, N, D, True, "int8", 64, "bhnd", cuda_dev)
    want = pa.backward_from_checkpoint(*kept, do, lse, seg)
    flat = torch.full((B * N * (Hq * D + 8) + 8,), 3.0, dtype=torch.bfloat16, device=cuda_dev)
    odd = flat[8:].as_strided((B, Hq, N, D), (N * (Hq * D + 8), D, Hq * D + 8, 1))
    odd.copy_(do)
    assert odd.data_ptr() % 32 == 16
    got = pa.backward_from_checkpoint(*kept, odd, lse, seg)
    n = pa.pa_bwd_ckpt_workspace_bytes(B, Hq, Hkv, N, D)
    ws = torch.empty(n + 16, dtype=torch.uint8, device=cuda_dev)[16:]
    assert ws.data_ptr() % 32 == 16
    again = pa.backward_from_checkpoint(*kept, do, lse, seg, ws=ws)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    for x, y, z in zip(want, got, again):
        assert torch.equal(x, y) and torch.equal(x, z)


@pytest.mark.parametrize("B,N", [(4100, 100), (1, 524_417), (2, 300_001)])
def test_backward_behind_the_tile_table_of_many_tiles(B, N, cuda_dev):
    """More than 4,096 tiles: the table and the work lists take a kernel each. dv
    has the bits of pa_bwd on the loaded tensors, dq and dk differ by out's
    rounding inside delta and dk's by P's; rows at both ends against the oracle."""
    Hq, Hkv, D = 2, 1, 64
    g = torch.Generator(device=cuda_dev).manual_seed(6)
    q, k, v, do = (torch.randn(B, H, N, D, generator=g, device=cuda_dev).bfloat16() for H in (Hq, Hkv, Hkv, Hq))
    lens = torch.randint(1, 200, (B, N // 90 + 2), generator=g, device=cuda_dev)
    seg = torch.searchsorted(lens.cumsum(1), torch.arange(N, device=cuda_dev).expand(B, N).contiguous(), right=True).int()
    out, lse = pa.forward(q, k, v, seg)
    kept = pa.checkpoint_save([q, k, v, out])
    ws = torch.empty(pa.pa_bwd_ckpt_workspace_bytes(B, Hq, Hkv, N, D), dtype=torch.uint8, device=cuda_dev)
    got = pa.backward_from_checkpoint(*kept, do, lse, seg, ws=ws)
    again = pa.backward_from_checkpoint(*kept, do, lse, seg)
    lq, lk, lv, lo = pa.checkpoint_load(kept)
    want = pa.backward(lq, lk, lv, lo, do, lse, seg)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    assert torch.equal(got[2], want[2]) and all(torch.equal(x, y) for x, y in zip(got, again))
    for x, y in zip(got, want):
        assert (x.float() - y.float()).norm() <= 2.0 ** -7 * x.float().norm()
    # whole segments at the start of the first row and the end of the last
    for b, last in ((0, False), (B - 1, True)):
        ids = seg[b].cpu().numpy()
        cut = np.flatnonzero(np.diff(ids)) + 1
        r = np.s_[cut[cut >= N - 400][0] if N > 400 else 0:] if last else np.s_[:(cut[cut <= 400][-1] if N > 400 else N)]
        sub = [pa.Checkpoint(c.codes[b:b + 1, :, r].contiguous(), c.scales[b:b + 1, :, r].contiguous(), c.block) for c in kept]
        w = _oracle(sub, do[b:b + 1, :, r], lse[b:b + 1, :, r], seg[b:b + 1, r], D)
        for x, y, n in zip(got, w, ("dq", "dk", "dv")):
            rel = np.linalg.norm(f64(x[b:b + 1, :, r]) - y) / np.linalg.norm(y)
            print(f"{n}: relL2 {rel:.2e}")
            assert rel <= TWO_ROUNDINGS, n


def test_backward_is_pa_bwds_on_what_a_load_gives(cuda_dev):
    """dv takes P and dout alone, so it has the bits of pa_bwd on the loaded
    tensors; dq and dk differ by out's rounding to bf16 inside delta."""
    q, k, v, do, seg, out, lse, kept = _case(1, 4, 2, 300, 128, True, "int8", 64, "bhnd", cuda_dev)
    lq, lk, lv, lo = pa.checkpoint_load(kept)
    a = pa.backward(lq, lk, lv, lo, do, lse, seg)
    b = pa.backward_from_checkpoint(*kept, do, lse, seg)
    assert torch.equal(a[2], b[2])
    for x, y in zip(a, b):
        assert (x.float() - y.float()).norm() <= 2.0 ** -7 * x.float().norm()


def test_backward_keeps_neighbours_and_captures(cuda_dev):
    """Gradients into slices leave what lies around them; a captured call
    replays to the same bits."""
    q, k, v, do, seg, out, lse, kept = _case(1, 2, 2, 200, 64, True, "int8", 64, "bnhd", cuda_dev)
    want = pa.backward_from_checkpoint(*kept, do, lse, seg)
    big = [torch.full((1, 260, 2, 64), 3.0, device=cuda_dev, dtype=torch.bfloat16) for _ in range(3)]
    views = [b[:, 30:230].transpose(1, 2) for b in big]
    do2 = torch.zeros_like(big[0])
    do2[:, 30:230] = do.transpose(1, 2)
    ws = torch.empty(pa.pa_bwd_ckpt_workspace_bytes(1, 2, 2, 200, 64), dtype=torch.uint8, device=cuda_dev)
    g = torch.cuda.CUDAGraph()
    pa.pa_bwd_ckpt(*kept, do2[:, 30:230].transpose(1, 2), lse, seg, *views, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pa.pa_bwd_ckpt(*kept, do2[:, 30:230].transpose(1, 2), lse, seg, *views, ws)
    for x in views:
        x.zero_()
    g.replay()
    torch.cuda.synchronize()
    for x, w, b in zip(views, want, big):
        assert torch.equal(x, w) and (b[:, :30] == 3).all() and (b[:, 230:] == 3).all()


def test_backward_refusals(cuda_dev):
    q, k, v, do, seg, out, lse, kept = _case(1, 2, 2, 128, 64, True, "int8", 64, "bhnd", cuda_dev)
    other = pa.checkpoint_save([q], format="e4m3")[0]
    with pytest.raises(ValueError):
        pa.backward_from_checkpoint(other, *kept[1:], do, lse, seg)
    with pytest.raises(ValueError):
        pa.backward_from_checkpoint(*kept, do[:, :1], lse, seg)
    with pytest.raises(ValueError):
        pa.backward_from_checkpoint(*kept, do, lse, seg.long())
    with pytest.raises(pa.PAError):
        pa.backward_from_checkpoint(*kept, do, lse, seg, ws=torch.empty(256, dtype=torch.uint8, device=cuda_dev))


# -------------------------------------------------------------- one step
def test_a_policy_step_over_packed_rows(cuda_dev):
    """The operators as a policy step uses them: attention forward on packed
    rows, its tensors kept in 8 bits, the log probabilities of the sampled
    tokens with an entropy bonus from the attention's output as hidden states,
    their gradient, and the attention backward from the 8-bit tensors, against
    the same chain in fp64 without the 8 bits.

    int8 in blocks of 64 normals keeps each element to a uniform error of
    scale / sqrt(12), scale = 2.5 sigma / 127: 0.6% of sigma. It enters the
    gradients through P (a relative error of the score's, 0.6% sqrt(2) of
    |s| ~ 1) and linearly through q, k and out: about 1% of the norm each, so
    within 5% together."""
    B, Hq, Hkv, N, D, V = 2, 4, 2, 200, 64, 700
    q, k, v = (_rows(9, 90 + i, B, H, N, D, "bnhd", cuda_dev) for i, H in enumerate((Hq, Hkv, Hkv)))
    ids = np.stack([synth.lengths_to_ids(synth.uniform_lengths(40 + b, N, 5, 60)) for b in range(B)]).astype(np.int32)
    seg = torch.from_numpy(ids).to(cuda_dev)
    head = torch.from_numpy(synth.bf16_normal(9, 95, (V, Hq * D)).view(np.int16)).view(torch.bfloat16).to(cuda_dev)
    t = (synth.uint64s(9, 96, B * N) % np.uint64(V)).astype(np.int32)
    t[ids.reshape(-1) == 0] = -1  # a prompt
    targets = torch.from_numpy(t).to(cuda_dev)
    adv = synth.normals(9, 97, B * N).astype(np.float32)
    g, e = torch.from_numpy(adv).to(cuda_dev), torch.full((B * N,), 0.1, device=cuda_dev)

    out, lse = pa.forward(q, k, v, seg)
    hidden = out.transpose(1, 2).reshape(B * N, Hq * D)
    kept = pa.checkpoint_save([q, k, v, out])
    hkept, = pa.checkpoint_save([hidden])
    logp, lse_v, ent, ids5, alt5 = pa.token_logprobs_forward(hidden, head, targets, temperature=8.0, top=5)
    dh, dw = pa.token_logprobs_backward(hkept, head, targets, lse_v, ent, g, e, temperature=8.0)
    dout = dh.view(B, N, Hq, D).transpose(1, 2)
    dq, dk, dv = pa.backward_from_checkpoint(*kept, dout, lse, seg)
    torch.cuda.synchronize()

    from oracle import logprobs
    o64, l64, _ = oracle.forward(f64(q), f64(k), f64(v), ids, 1 / math.sqrt(D))
    h64 = o64.transpose(0, 2, 1, 3).reshape(B * N, Hq * D)
    elogp, _, eent, _, _ = logprobs.forward(h64, f64(head), t, 8.0)
    assert np.abs(logp.cpu().numpy() - elogp).max() < 0.1 and np.abs(ent.cpu().numpy() - eent).max() < 0.1
    edh, edw = logprobs.backward(h64, f64(head), t, adv, np.full(B * N, np.float32(0.1)), 8.0)
    ed = edh.reshape(B, N, Hq, D).transpose(0, 2, 1, 3)
    want = oracle.attention(f64(q), f64(k), f64(v), ids, 1 / math.sqrt(D), ed)
    for x, y, n in ((dh, edh, "dhidden"), (dw, edw, "dhead"), (dq, want["dq"], "dq"), (dk, want["dk"], "dk"),
                    (dv, want["dv"], "dv")):
        rel = np.linalg.norm(f64(x) - y) / np.linalg.norm(y)
        print(f"{n}: relL2 {rel:.2e}")
        assert rel <= 0.05, n
