"""The Python binding's objects around the paged cache and the rotation, on the host
(no GPU needed)."""
import copy
import ctypes
import pickle

import pytest
import torch

import segment_masked_causal_gb300 as pa


@pytest.fixture(scope="module", autouse=True)
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


@pytest.mark.parametrize("D", [64, 96, 128])
def test_a_new_workspace_has_no_status(D, monkeypatch):
    """A step without rows launches nothing that would set the status word."""
    monkeypatch.setattr(torch, "empty", lambda n, **kw: torch.full((n,), 0xA5, **kw))  # memory that was used before
    k = torch.zeros(2, 2, 16, D, dtype=torch.bfloat16)
    ws = pa.paged_workspace(torch.zeros(0, 4, D, dtype=torch.bfloat16), pa.PagedCache(k, k))
    assert ws.numel() == pa.pa_paged_workspace_bytes(D) and ws.dtype == torch.uint8
    assert ws[:4].tolist() == [0] * 4 and ws[4] == 0xA5


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle", "module"])
@pytest.mark.parametrize("kw", [{}, dict(interleaved=True, amplitude=0.7), dict(scaling="bands", factor=4.0, original=2048),
                                dict(frequencies=[1.0, 1e-3, -0.25, 7.5] * 4)])
def test_a_rotary_is_copied_and_pickled(how, kw):
    """As a model that holds one is."""
    class Layer(torch.nn.Module):
        def __init__(self, rotary):
            super().__init__()
            self.rotary = rotary
    r = pa.Rotary(32, **kw)
    s = {"copy": lambda: copy.copy(r), "deepcopy": lambda: copy.deepcopy(r), "pickle": lambda: pickle.loads(pickle.dumps(r)),
         "module": lambda: copy.deepcopy(Layer(r)).rotary}[how]()
    assert s is not r and s.c is not r.c and bytes(s.c) == bytes(r.c)
    assert (s.rot, s.interleaved, s.amplitude, s.frequencies) == (r.rot, r.interleaved, r.amplitude, r.frequencies)
    assert ctypes.addressof(s.ref._obj) == ctypes.addressof(s.c)
