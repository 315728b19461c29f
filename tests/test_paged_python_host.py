"""The Python binding's objects around the paged cache and the rotation, on the host
(no GPU needed)."""
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
