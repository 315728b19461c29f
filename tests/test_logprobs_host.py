"""Token log probabilities on the host: the fp64 oracle's pins and the C ABI's
refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

import segment_masked_causal_gb300 as pa
from oracle import logprobs

FAKE = 0x100000  # a 16-byte-aligned non-null address; never dereferenced on refusal


@pytest.fixture(scope="module")
def L():
    from segment_masked_causal_gb300 import build
    build.build()
    return pa.lib()


def _case(seed, N=5, V=11, D=7):
    r = np.random.default_rng(seed)
    t = r.integers(0, V, N)
    t[1] = -1
    return r.normal(size=(N, D)), r.normal(size=(V, D)), t, r.normal(size=N), r.normal(size=N)


@pytest.mark.parametrize("T", [1.0, 0.7, 2.0])
def test_oracle_against_autograd(T):
    H, W, t, g, e = _case(1)
    h, w = (torch.tensor(x, requires_grad=True) for x in (H, W))
    lp = torch.log_softmax(h @ w.T / T, 1)
    scored = torch.tensor(t >= 0)
    logp = torch.where(scored, lp[torch.arange(5), torch.tensor(t).clamp(min=0)], torch.zeros(()).double())
    ent = -(lp.exp() * lp).sum(1)
    (torch.tensor(g) * logp + torch.tensor(e) * ent).sum().backward()
    got = logprobs.forward(H, W, t, T, top=3)
    # fp64 on both sides: a few hundred roundings of 2^-53 on values below 10
    assert np.abs(got[0] - logp.detach().numpy()).max() < 1e-12
    assert np.abs(got[2] - ent.detach().numpy()).max() < 1e-12
    assert (got[3] == torch.topk(lp, 3).indices.numpy()).all()
    dH, dW = logprobs.backward(H, W, t, g, e, T)
    assert np.abs(dH - h.grad.numpy()).max() < 1e-12 and np.abs(dW - w.grad.numpy()).max() < 1e-12


def test_oracle_against_differences():
    """Central differences: the error is h^2 / 6 of the third derivative (of
    order 10 here) plus 2^-53 / h, at h = 1e-5 below 1e-9."""
    H, W, t, g, e = _case(2)
    loss = lambda H, W: (lambda r: (g * r[0] * (t >= 0) + e * r[2]).sum())(logprobs.forward(H, W, t, 0.8))
    dH, dW = logprobs.backward(H, W, t, g, e, 0.8)
    h = 1e-5
    for A, dA, f in ((H, dH, lambda x: loss(x, W)), (W, dW, lambda x: loss(H, x))):
        for i in np.ndindex(A.shape):
            up, dn = A.copy(), A.copy()
            up[i] += h
            dn[i] -= h
            assert abs((f(up) - f(dn)) / (2 * h) - dA[i]) < 1e-8


def test_oracle_uniform_ties_and_one_entry():
    H, W = np.zeros((2, 4)), np.ones((6, 4))
    logp, lse, ent, ids, alt = logprobs.forward(H, W, [3, 6], top=4)
    assert np.allclose(logp, [-np.log(6), 0.0]) and np.allclose(ent, np.log(6))
    assert (ids == [0, 1, 2, 3]).all() and np.allclose(alt, -np.log(6))
    logp, lse, ent, ids, alt = logprobs.forward(np.ones((1, 4)), W[:1], [0], top=1)
    assert logp[0] == 0 and ent[0] == 0 and ids[0, 0] == 0


def test_forward_refusals(L):
    need = L.pa_logp_workspace_bytes(256, 1000, 128, 8)
    assert need > 0
    for bad in ((0, 1000, 128, 0), (256, 0, 128, 0), (256, 1000, 96, 0), (256, 1000, 128, 33), (256, 1000, 128, -1),
                (256, 20, 128, 21), ((1 << 30) + 1, 1000, 128, 0), (256, 1000, 16448, 0)):
        assert L.pa_logp_workspace_bytes(*bad) == 0

    def f(N=256, V=1000, D=128, T=1.0, top=8, h=FAKE, w=FAKE, t=FAKE, lp=FAKE, ent=FAKE, ids=FAKE, alt=FAKE, ws=FAKE,
          n=1 << 30):
        return L.pa_logp_fwd(N, V, D, T, top, h, w, t, lp, FAKE, ent, ids, alt, ws, n, None)
    assert f(N=0) == 4 and f(V=0) == 4 and f(D=96) == 4 and f(top=33) == 4 and f(V=7) == 4
    for T in (0.0, -1.0, float("inf"), float("nan"), 1e-45):
        assert f(T=T) == 4
    assert f(h=None) == 1 and f(ent=None) == 1 and f(ws=None) == 1 and f(ids=None) == 1 and f(alt=None) == 1
    assert f(w=FAKE + 8) == 5 and f(t=FAKE + 4) == 5 and f(alt=FAKE + 4) == 5 and f(ws=FAKE + 8) == 5
    assert f(n=need - 1) == 6
    if not torch.cuda.is_available():
        assert f() in (7, 8)
        assert f(top=0, ids=None, alt=None) in (7, 8)  # no alternatives: their pointers are not used


def test_backward_refusals(L):
    need = L.pa_logp_bwd_workspace_bytes(256, 1000, 128)
    assert need > 0 and L.pa_logp_bwd_workspace_bytes(256, 1000, 100) == 0

    def f(N=256, D=128, T=1.0, lse=FAKE, ent=FAKE, g=FAKE, e=FAKE, dh=FAKE, dw=FAKE, ws=FAKE, n=need):
        return L.pa_logp_bwd(N, 1000, D, T, FAKE, FAKE, FAKE, lse, ent, g, e, dh, dw, ws, n, None)
    assert f(N=0) == 4 and f(D=32) == 4 and f(T=0.0) == 4
    assert f(lse=None) == 1 and f(g=None) == 1 and f(dh=None) == 1 and f(ent=None) == 1
    assert f(dw=FAKE + 8) == 5 and f(e=FAKE + 4) == 5 and f(g=FAKE + 4) == 5
    assert f(n=need - 1) == 6
    if not torch.cuda.is_available():
        assert f() in (7, 8)
        assert f(ent=None, e=None, dw=None) in (7, 8)


def test_python_refusals():
    h, w, t = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(9, 64, dtype=torch.bfloat16), torch.zeros(4).int()
    with pytest.raises(ValueError, match="head"):
        pa.token_logprobs_forward(h, w[:, :32], t)
    with pytest.raises(ValueError, match="targets"):
        pa.token_logprobs_forward(h, w, t[:3])
    with pytest.raises(pa.PAError):
        pa.token_logprobs_forward(h, w, t, top=10)
    f = torch.zeros(4)
    with pytest.raises(ValueError, match="g_entropy"):
        pa.pa_logp_bwd(h, w, t, f, f, f, f[:2], h, w, f)


def _splits(N, V, slots=152):
    """The split rule restated: what the launch takes for `slots` SMs."""
    TM, U = -(-N // 128), -(-V // 32)
    most = max(1, min(160, U, 2432 // TM))
    best = None
    for s in range(1, most + 1):
        per = -(-U // s)
        used = -(-U // per)
        cost = -(-TM * used // slots) * (per + 8)
        if best is None or cost < best[0]:
            best = (cost, used, per)
    return best[1], best[2], most


@pytest.mark.parametrize("N", [1, 2, 127, 128, 129, 1000, 8192, 100000])
@pytest.mark.parametrize("V", [1, 31, 33, 1000, 32003, 151936])
def test_splits_cover_the_vocabulary_within_the_workspace(N, V, L):
    """Every unit of 32 rows lies in one split, none is empty, and the partial
    results (16 bytes a token and split, 8 for each alternative) fit."""
    used, per, most = _splits(N, V)
    U = -(-V // 32)
    assert used <= most and (used - 1) * per < U <= used * per
    for top in (0, min(V, 32)):
        assert L.pa_logp_workspace_bytes(N, V, 64, top) >= 256 + used * N * (16 + 8 * top)


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 128, 129, 1000, 4096, 100_000, 1 << 18])
@pytest.mark.parametrize("V", [1, 32003, 540_001, 1_100_000, 1 << 25, 1 << 30])
def test_backward_workspace_is_bounded(N, V, L):
    """One chunk's dz takes 128 MiB at most and its transposed copy, whose rows
    are whole runs of 64 tokens, 256 MiB; beside them dH's accumulators, one for
    each of up to 64 runs of the contraction (the D = 64 of them here)."""
    assert 0 < L.pa_logp_bwd_workspace_bytes(N, V, 64) <= (384 << 20) + 64 * N * 64 * 4 + 4096


@pytest.mark.parametrize("sms", [1, 2, 3, 66, 148, 152, 160])
@pytest.mark.parametrize("N", [1, 8, 32, 33, 64, 65, 127, 128, 129, 256, 257, 777, 1500, 8192, 100_000, 1 << 30])
def test_the_forwards_plan_covers_the_vocabulary(N, sms, L):
    """What the launch takes: every unit of 32 rows lies in one split and none is
    empty; tiles are 1 to 8 units wide and none of a split's is empty; the splits'
    partial results (16 bytes a token, 8 for each alternative) fit the workspace,
    and a token's lists the 40 KB of shared memory that the merge gives them."""
    for V in (1, 31, 32, 33, 255, 256, 257, 1000, 5003, 32003, 50257, 151936, 1_000_001, 1 << 25, 1 << 30):
        for D in (64, 128, 512, 4096, 16384):
            pair, splits, per, width = pa.pa_logp_plan(N, V, D, sms)
            U = -(-V // 32)
            assert 1 <= splits <= 160 and (splits - 1) * per < U <= splits * per
            assert 1 <= width <= 8 and width <= per and per - (-(-per // width) - 1) * width >= 1
            assert not pair or (N > 128 and sms >= 2)
            for top in (0, min(V, 32)):
                assert L.pa_logp_workspace_bytes(N, V, D, top) >= 256 + splits * N * (16 + 8 * top)
                assert splits * top * 8 <= 40960


def test_plan_refusals(L):
    out = (ctypes.c_int32 * 4)()
    assert L.pa_logp_plan(0, 10, 64, 152, out) == 4 and L.pa_logp_plan(1, 10, 65, 152, out) == 4
    assert L.pa_logp_plan(1, 10, 64, 0, out) == 4 and L.pa_logp_plan(1, 10, 64, 152, None) == 1
    assert L.pa_logp_plan(1, 10, 64, 152, out) == 0
