"""Rotary positions at any 32-bit position, to the bound of near ones: the part of the angle
that a far position adds, 2^-32 turns (1.5e-9 radians), is inside the 4 * 2^-24 of
test_gpu_rotary.py's derivation (pi/4 * 2^-24 + 2^-23 + 2^-24 = 3.8 * 2^-24)."""
import numpy as np
import pytest
import torch

import segment_masked_causal_gb300 as pa
import synth
from oracle import rotary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


@pytest.mark.parametrize("theta", [1e4, 5e5])
@pytest.mark.parametrize("interleaved,backward", [(False, False), (True, True)])
def test_far_positions_are_as_exact_as_near_ones(cuda_dev, theta, interleaved, backward):
    r = pa.Rotary(128, theta=theta, interleaved=interleaved)
    pos = np.concatenate([[0, 1, 2 ** 28, 2 ** 31 - 1, -1, -2 ** 31], (synth.uint64s(3, 82, 250) >> np.uint64(32)).astype(np.uint32).view(np.int32)])
    N = len(pos)
    x = synth.normals(4, 83, 2 * N * 128).reshape(1, 2, N, 128).astype(np.float32)
    f = pa.rotary_backward if backward else pa.rotary_forward
    y = f([torch.from_numpy(x).to(cuda_dev)], r, torch.from_numpy(pos.astype(np.int32)[None]).to(cuda_dev))[0]
    X = x.astype(np.float64)
    want = rotary.rotate(X, pos[None, None], r.frequencies, interleaved=interleaved, backward=backward)
    assert (np.abs(y.double().cpu().numpy() - want) <= 2.0 ** -21 * rotary.weight(X, r.frequencies, interleaved)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("bad", ["address", "strides", "gap", "heads"])
def test_a_list_of_several_launches_is_turned_whole_or_not_at_all(cuda_dev, dtype, bad):
    r = pa.Rotary(64)
    xs = [torch.randn(2, 3, 5, 64, device=cuda_dev).to(dtype) for _ in range(6)]
    keep = [x.clone() for x in xs]
    wide = torch.randn(2, 3, 5, 80, device=cuda_dev).to(dtype)
    last = {"address": wide[..., 2:66], "strides": wide.flatten()[:2 * 3 * 5 * 66].view(2, 3, 5, 66)[..., :64],
            "gap": wide.flatten().as_strided((2, 3, 5, 64), (960, 320, 48, 1)), "heads": wide[:, :0, :, :64]}[bad]
    kept = wide.clone()
    with pytest.raises(pa.PAError, match="PA_ERR_ALIGN" if bad in ("address", "strides") else "PA_ERR_SHAPE"):
        pa.rotary_forward(xs + [last], r, out=xs + [last])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(xs, keep)) and torch.equal(wide, kept)
    with pytest.raises(pa.PAError):  # alone it is refused as well
        pa.rotary_forward([last], r, out=[last])
    turned = pa.rotary_forward(xs, r, out=xs)
    assert all(torch.equal(a, pa.rotary_forward([b], r)[0]) for a, b in zip(turned, keep))
