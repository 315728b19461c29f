"""Rotary positions on the GPU against the fp64 oracle.

An angle is a 32-bit fraction of a turn, off by 2^-32 turns (1.5e-9 radians), the part
of it past the nearest quarter, at most pi/4, rounded to fp32: 2^-24 * pi/4. Sine and
cosine are within 2^-23 and the amplitude's product within 2^-24 of themselves, so c and
s are within 4 * 2^-24 a of theirs. An element is the sum of two such products (|x1| +
|x2|) a = w: 4 * 2^-24 w from the factors and 2 * 2^-24 w from the product and the sum,
below 2^-21 w together; a bf16 result is off by its rounding, 2^-8 of itself, as well."""
import numpy as np
import pytest
import torch

import oracle
import segment_masked_causal_gb300 as pa
import synth
from oracle import rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def normals(shape, seed, dev, dtype):
    return torch.from_numpy(synth.normals(seed, 80, int(np.prod(shape))).reshape(shape)).to(dtype).to(dev)


def memory(x, order):
    """The (B, H, N, D) values of x in another memory order."""
    if order == "bnhd":
        return x.transpose(1, 2).contiguous().transpose(1, 2)
    if order == "sliced":  # heads of a wider projection, rows with a gap behind them
        B, H, N, D = x.shape
        wide = torch.full((B, N, H + 2, D + 8), float("nan"), dtype=x.dtype, device=x.device)
        view = wide[:, :, 1:H + 1, :D].transpose(1, 2)
        view.copy_(x)
        return view
    return x


def check(got, x, pos, r, backward=False):
    X = f64(x)
    want = rotary.rotate(X, pos[:, None], r.frequencies, r.amplitude, r.interleaved, backward)
    w = rotary.weight(X, r.frequencies, r.interleaved) * abs(r.amplitude)
    tol = 2.0 ** -21 * w + (2.0 ** -8 * np.abs(want) if got.dtype == torch.bfloat16 else 0)
    err = np.abs(f64(got) - want)
    assert got.dtype == x.dtype and got.shape == x.shape
    assert (err <= tol).all(), (err - tol).max()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(64, 64), (96, 24), (96, 96), (128, 128), (128, 8), (128, 40), (72, 64), (256, 128), (8, 8)])
@pytest.mark.parametrize("order", ["bhnd", "bnhd", "sliced"])
def test_against_oracle(cuda_dev, dtype, interleaved, D, rot, order):
    B, N = 2, 37
    r = pa.Rotary(rot, interleaved=interleaved, amplitude=1.25)
    xs = [memory(normals((B, H, N, D), 3 + H, cuda_dev, dtype), order) for H in (5, 1)]
    pos = (synth.uint64s(9, 81, B * N) % np.uint64(100000)).astype(np.int32).reshape(B, N)
    p = torch.from_numpy(pos).to(cuda_dev)
    for x, y, dx in zip(xs, pa.rotary_forward(xs, r, p), pa.rotary_backward(xs, r, p)):
        check(y, x, pos, r)
        check(dx, x, pos, r, backward=True)


@pytest.mark.parametrize("pos", [0, 1, 2 ** 20 + 3, 2 ** 31 - 1, -1, -2 ** 31])
def test_far_positions(cuda_dev, pos):
    r = pa.Rotary(128, theta=5e5)
    x = normals((1, 3, 1, 128), 5, cuda_dev, torch.float32)
    at = np.full((1, 1), pos, np.int32)
    y = pa.rotary_forward([x], r, torch.from_numpy(at).to(cuda_dev))[0]
    # the frequency in turns is a double: 2^-53 of a turn count of up to 2^31 / 2 pi on top
    X, want = f64(x), rotary.rotate(f64(x), at[:, None], r.frequencies)
    w = rotary.weight(X, r.frequencies)
    assert (np.abs(f64(y) - want) <= w * (2.0 ** -21 + abs(pos) * 2.0 ** -51)).all()


def test_default_positions_lists_and_in_place(cuda_dev):
    B, N, D = 2, 130, 64
    r = pa.Rotary(32)
    xs = [normals((B, H, N, D), 20 + H, cuda_dev, torch.bfloat16) for H in (1, 2, 3, 4, 5, 17)]  # two launches
    p = torch.arange(N, device=cuda_dev, dtype=torch.int32).expand(B, N).contiguous()
    a, b = pa.rotary_forward(xs, r), pa.rotary_forward(xs, r, p)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    keep = [x.clone() for x in xs]
    assert pa.rotary_forward(xs, r, p, out=xs) == xs
    assert all(torch.equal(u, v) for u, v in zip(a, xs))
    # there and back: two roundings
    back = pa.rotary_backward(xs, r, p)
    assert all((u - v).abs().max() <= 2 ** -6 * v.abs().max() for u, v in zip(back, keep))
    assert torch.equal(xs[0][..., 32:], keep[0][..., 32:])
    assert pa.rotary_forward([], r) == []


@pytest.mark.parametrize("heads,N", [(1, 1), (1, 5000), (200, 3), (40, 700)])
def test_many_and_few(cuda_dev, heads, N):
    r = pa.Rotary(128)
    x = normals((1, heads, N, 128), 6, cuda_dev, torch.bfloat16)
    check(pa.rotary_forward([x], r)[0], x, np.arange(N)[None], r)


@pytest.mark.parametrize("B,N,runs", [(1, 1, "one"), (3, 1000, "short"), (2, 1025, "one"), (1, 8192, "packed"),
                                      (1, 70001, "one"), (2, 9001, "long"), (1, 5000, "each")])
def test_positions(cuda_dev, B, N, runs):
    rng = np.random.default_rng(N)
    seg = np.zeros((B, N), np.int32)
    for b in range(B):
        top = {"one": N, "short": 9, "packed": 2048, "long": 6000, "each": 1}[runs]
        n, i = 0, 0
        while n < N:
            step = top if runs in ("one", "each") else int(rng.integers(1, top + 1))
            seg[b, n:n + step] = (i % 3) - 1  # ids that come back
            n, i = n + step, i + 1
    got = pa.segment_positions(torch.from_numpy(seg).to(cuda_dev))
    assert got.dtype == torch.int32 and (got.cpu().numpy() == rotary.positions(seg)).all()


def test_captured_and_replayed_on_another_stream(cuda_dev):
    r = pa.Rotary(64, interleaved=True)
    x = normals((2, 4, 300, 64), 7, cuda_dev, torch.bfloat16)
    seg = torch.from_numpy(np.repeat(np.arange(4, dtype=np.int32), 75)[None].repeat(2, 0)).to(cuda_dev)
    y = torch.empty_like(x)
    pos = torch.empty_like(seg)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        pa.pa_positions(seg, pos)
        pa.pa_rope([x], [y], r, pos)
    for k in range(2):
        x.normal_()
        seg.copy_(torch.arange(300, device=cuda_dev, dtype=torch.int32) // (50 + 31 * k))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, pa.rotary_forward([x], r, pa.segment_positions(seg))[0])


def test_python_refusals(cuda_dev):
    r = pa.Rotary(32)
    x = torch.zeros(2, 3, 5, 64, device=cuda_dev)
    for bad, match in (([x, x.bfloat16()], "type"), ([x, x[:1]], "one B, N and D"), ([x[0]], r"\(B, H, N, D\)"),
                       ([x, x.cpu()], "current CUDA device"), ([x.transpose(2, 3)], "last dim"), ([x.half()], "bfloat16")):
        with pytest.raises(ValueError, match=match):
            pa.rotary_forward(bad, r, out=[torch.empty_strided(b.shape, b.stride(), dtype=b.dtype, device=b.device) for b in bad])
    with pytest.raises(ValueError, match="positions"):
        pa.rotary_forward([x], r, torch.zeros(2, 4, dtype=torch.int32, device=cuda_dev))
    with pytest.raises(ValueError, match="positions"):
        pa.rotary_forward([x], r, torch.zeros(2, 5, dtype=torch.int64, device=cuda_dev))
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.rotary_forward([x], r, torch.zeros(2, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="one output"):
        pa.rotary_forward([x], r, out=[])
    with pytest.raises(pa.PAError, match="PA_ERR_SHAPE"):
        pa.rotary_forward([x[..., :16].contiguous()], r)  # narrower than rot
    with pytest.raises(ValueError, match="seg"):
        pa.segment_positions(torch.zeros(2, 4, dtype=torch.int64, device=cuda_dev))


def test_rotary_attention_and_gradients_on_packed_rows(cuda_dev):
    """Positions, rotation, attention and the way back, against the oracle's
    attention on the rotated tensors and the oracle's rotation of its gradients."""
    w = synth.workload("tiny_3seg")
    t = w.tensors()
    to = lambda b: torch.from_numpy(np.ascontiguousarray(b).view(np.int16)).view(torch.bfloat16).to(cuda_dev)
    q, k, v, do = (to(t[x]) for x in ("q", "k", "v", "do"))
    seg = torch.from_numpy(w.seg).to(cuda_dev)
    r = pa.Rotary(q.shape[-1])
    pos = pa.segment_positions(seg)
    qr, kr = pa.rotary_forward([q, k], r, pos)
    out, lse = pa.forward(qr, kr, v, seg)
    dqr, dkr, dv = pa.backward(qr, kr, v, out, do, lse, seg)
    dq, dk = pa.rotary_backward([dqr, dkr], r, pos)
    ref = oracle.attention(f64(qr), f64(kr), f64(v), w.seg, w.scale, f64(do))
    P = rotary.positions(w.seg)[:, None]
    assert np.abs(f64(out) - ref["o"]).max() <= 1e-2
    for got, want in ((dq, rotary.rotate(ref["dq"], P, r.frequencies, backward=True)),
                      (dk, rotary.rotate(ref["dk"], P, r.frequencies, backward=True)), (dv, ref["dv"])):
        assert np.linalg.norm(f64(got) - want) <= 2e-2 * np.linalg.norm(want)
