"""Token log probabilities on the GPU against the fp64 oracle.

Hidden states and head lie on grids (multiples of 1/8 and of a power of two),
so that every logit is exact in fp32 whatever the order of its sum: the
alternatives' order, ties included, has to be the oracle's, and the
tolerances below count only what the epilogue does.

With Z = max |z| (after the temperature) in nats:
  t = z log2 e - m    the factor log2(e)/T is off by 2^-24, the fused product
                      rounds once: |dt| <= 2^-24 (1.45 Z) + 2^-24 (2 * 1.45 Z)
  2^t                 2^-22 from the exponential, so each term is within
                      r = ln 2 * |dt| + 2^-22 of itself
  S                   a split's sum runs over at most V / 32 chunk sums, each
                      of 16 pairwise-packed terms: 2^-24 (V / 32 + 32) more
so lse is within r + 2^-24 (V / 32 + 32) plus a few roundings of itself, logp
adds one of the logit's, and the entropy, whose sum takes |t| <= L = H + ln V
+ 1 in the mean, within (2 + L) times that."""
import math

import numpy as np
import pytest
import torch

import segment_masked_causal_gb300 as pa
import synth
from oracle import logprobs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


def grid(seed, stream, shape, most, step):
    """Uniform integers in [-most, most] times step, fp64."""
    u = synth.uint64s(seed, stream, int(np.prod(shape)))
    return ((u % np.uint64(2 * most + 1)).astype(np.float64) - most).reshape(shape) * step


def inputs(N, V, D, seed):
    H = grid(seed, 60, (N, D), 15, 1 / 8)  # std 1.1
    W = grid(seed, 61, (V, D), 15, 2.0 ** -round(math.log2(4 * math.sqrt(D))))  # logits of std 2 to 4
    t = (synth.uint64s(seed, 62, N) % np.uint64(V)).astype(np.int32)
    if N > 3:
        t[1], t[3] = -1, V  # not scored
    return H, W, t


def dev_bf16(x, dev):
    b = torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)
    assert (b.double().numpy() == x).all() or not np.isfinite(x).all()
    return b.to(dev)


def run(H, W, t, dev, T=1.0, top=0):
    h, w, tt = dev_bf16(H, dev), dev_bf16(W, dev), torch.from_numpy(t).to(dev)
    ws = torch.empty(pa.pa_logp_workspace_bytes(h.shape[0], w.shape[0], h.shape[1], top), dtype=torch.uint8, device=dev)
    got = pa.token_logprobs_forward(h, w, tt, temperature=T, top=top, ws=ws)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    return [None if g is None else g.cpu().numpy() for g in got]


def check(got, want, V, Z):
    logp, lse, ent, ids, alt = (None if g is None else g.astype(np.float64) for g in got)
    e_logp, e_lse, e_ent, e_ids, e_alt = want
    u = 2.0 ** -24
    r = 3 * 1.45 * Z * u + 4 * u + u * (V / 32 + 32)
    bar = r + 4 * u * (np.abs(e_lse) + Z)
    for g, e, n in ((logp, e_logp, "logp"), (lse, e_lse, "lse")):
        err = np.abs(g - e)
        print(f"{n}: max err {err.max():.2e} of {bar.min():.2e}")
        assert (err <= bar).all(), n
    L = e_ent + math.log(V) + 1
    err = np.abs(ent - e_ent)
    print(f"entropy: max err {err.max():.2e}, relative to its bar {(err / (bar * (2 + L))).max():.2e}")
    assert (err <= bar * (2 + L)).all() and (ent >= 0).all()
    if ids is not None:
        assert (ids == e_ids).all()
        assert (np.abs(alt - e_alt) <= bar[:, None]).all()


CASES = [
    # one token and few; every row an alternative; a vocabulary of one and of
    # part of a unit; ragged everything over many splits; several token tiles;
    # the 32-slot and the 8-slot lists; the ring wraps
    (1, 33, 64, 1, 1.0), (1, 1000, 128, 5, 1.0), (3, 32, 64, 32, 1.0), (5, 8, 64, 8, 0.5), (2, 1, 64, 1, 1.0),
    (128, 31, 64, 3, 1.0), (130, 1003, 192, 8, 0.7), (300, 5000, 256, 20, 1.3), (257, 2049, 64, 0, 1.0),
    (33, 20011, 1024, 9, 1.0), (1, 40000, 512, 32, 1.0), (1000, 700, 640, 2, 2.0),
]


@pytest.mark.parametrize("N,V,D,top,T", CASES)
def test_forward_matches_oracle(N, V, D, top, T, cuda_dev):
    H, W, t = inputs(N, V, D, 7 * N + V)
    got = run(H, W, t, cuda_dev, T, top)
    want = logprobs.forward(H, W, t, T, top)
    if top == 0:
        assert got[3] is None and got[4] is None
    check(got, want, V, np.abs(H @ W.T).max() / T)


def on_device(H, W, t, T, top, dev):
    """The oracle's forward in fp64 on the device, for sizes that take the host long."""
    h, w, tt = (torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in (H, W, t))
    got = [[] for _ in range(5)]
    for a in range(0, len(t), 256):
        raw = h[a:a + 256] @ w.T
        lp = torch.log_softmax(raw / T, 1)
        ti = tt[a:a + 256].long()
        scored = (ti >= 0) & (ti < len(W))
        logp = lp.gather(1, torch.where(scored, ti, 0)[:, None])[:, 0]
        ids = torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :top]
        for g, x in zip(got, (torch.where(scored, logp, 0.0), torch.logsumexp(raw / T, 1), -(lp.exp() * lp).sum(1), ids,
                              lp.gather(1, ids))):
            g.append(x.cpu().numpy())
    return [np.concatenate(g) for g in got], (h @ w.T).abs().max().item() / T


# Pairs of CTAs with lists of 8, 16, 24 and 32 slots over several tiles of a split
# (both accumulators, each used again); single CTAs whose tile holds the tokens
# once, twice and four times; merges with fewer than eight tokens a block (more
# than 304 tokens with more than 640 entries each)
LISTS = [
    # N, V, D, top, pairs, least tiles of a split, merge with fewer tokens a block
    (1500, 20_000, 128, 8, True, 7, False), (700, 30_011, 128, 16, True, 5, False), (257, 151_936, 128, 3, False, 12, False),
    (400, 30_000, 64, 24, True, 4, True), (1000, 50_257, 256, 32, True, 11, False), (310, 60_000, 64, 20, False, 5, True),
    (600, 50_257, 64, 5, False, 7, False), (128, 151_936, 64, 12, False, 4, False), (70, 90_001, 64, 20, False, 3, False),
    (100, 90_001, 64, 8, False, 3, False), (40, 90_001, 64, 20, False, 3, False), (64, 90_001, 64, 32, False, 3, False),
    (20, 140_000, 64, 9, False, 4, False),
]


def planned(N, V, D, top, pair, tiles, small_merge):
    """That the launch takes the form the case is there for, on 152 SMs."""
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        return
    is_pair, splits, per, width = pa.pa_logp_plan(N, V, D)
    assert is_pair == pair and -(-per // width) >= tiles and (N > 304 and splits * top > 640) == small_merge


@pytest.mark.parametrize("case", LISTS, ids=lambda c: "-".join(map(str, c[:4])))
@pytest.mark.parametrize("order", ["random", "ties", "rising", "falling"])
def test_alternatives_over_tiles_splits_and_pairs(case, order, cuda_dev):
    """Random logits; a head whose rows come again and again, so that equal logits
    lie in other chunks, tiles and splits; logits that rise along the vocabulary,
    where every column enters the list, and that fall."""
    N, V, D, top = case[:4]
    planned(*case)
    H, W, t = inputs(N, V, D, N + V + top)
    if order == "ties":
        W = W[np.arange(V) % 911]
    elif order in ("rising", "falling"):
        # z = s v, s = +-2^-12: exact, since v = 1024 a + 4 b + c with a, b, c of eight bits
        H[:], W[:] = 0, 0
        v = np.arange(V)
        W[:, 0], W[:, 1], W[:, 2] = v // 1024, v // 4 % 256, v % 4
        H[:, :3] = np.array([0.25, 2.0 ** -10, 2.0 ** -12])
        H[(np.arange(N) % 5 == 0) ^ (order == "falling")] *= -1
    T = 1.0 if order != "ties" else 0.7
    got = run(H, W, t, cuda_dev, T, top)
    want, Z = on_device(H, W, t, T, top, cuda_dev)
    check(got, want, V, Z)


def test_ties_and_uniform_logits(cuda_dev):
    """Zero states make every logit equal: the lowest rows win, the entropy is
    ln V. Rows of the head that repeat tie exactly."""
    N, V, D = 40, 3001, 64
    H, W, t = inputs(N, V, D, 5)
    H[:7] = 0
    W[2000:] = W[:1001]
    for top in (6, 32):
        got = run(H, W, t, cuda_dev, 1.0, top)
        assert (got[3][:7] == np.arange(top)).all()
        check(got, logprobs.forward(H, W, t, 1.0, top), V, np.abs(H @ W.T).max())


def test_a_sure_token(cuda_dev):
    """One logit far above the rest: logp is the little that the others add,
    the entropy is tiny and not negative."""
    N, V, D = 3, 500, 64
    H, W = np.zeros((N, D)), np.zeros((V, D))
    H[0, 0], H[1, 0], H[2, 0] = 8, 16, 120
    W[77, 0] = 1
    got = run(H, W, np.array([77, 77, 77], np.int32), cuda_dev, 1.0, 2)
    want = logprobs.forward(H, W, [77] * 3, 1.0, 2)
    check(got, want, V, 120)
    assert (got[3] == [[77, 0]] * 3).all()
    # with 500 exp(-120) beside it S is 1 within half a step of fp32: log2 S and t
    # are off by 2^-23 together
    assert abs(got[2][2]) <= 2.0 ** -22 and abs(got[0][2]) <= 2.0 ** -22


# A token of logit a at its dominant row and -a at the V - 1 others, with g = 2a / T
# the gap in nats: S = 1 + tail, tail = (V - 1) exp(-g), so
#   logp = -ln(1 + tail), entropy = ln(1 + tail) + g tail / (1 + tail).
# In units of 2^-24 the sum S, which lies in [1, 2), loses at most half a step (one
# unit) in each addition on the way of the large term: 16 inside its own chunk of
# 32 columns, one at the split's end, 3 where the columns are shared by four warps,
# 9 in the merge; the exponential of the dominant term itself is within 2^-22 of 1
# (4 units). What the additions between the chunks lose is kept beside the sum. The
# small terms are each off by ln 2 * 2^-24 (3 * 1.45 a / T) for the argument and 2^-22
# for the exponential, and so is their sum A = sum 2^t t, which loses 16 + 3 + 9
# units of itself in additions, relative to |A| = g tail. So logp is within
# 40 (1 + tail) units, and the entropy within 40 + 80 (1 + g) tail (tail <= 1).
def check_dominant(N, V, T, dev):
    D = 64
    amp = np.arange(8 * 16, 12 * 16 + 1) / 16 * T  # gaps of 16 to 24
    amp = np.round(amp * 16) / 16
    first = [0, V // 3, V - 1, 31]  # the dominant row, by the token's column
    a = amp[(np.arange(N) * 37) % len(amp)]
    g = 2 * a / T
    tail = (V - 1) * np.exp(-g)
    a = np.where(tail <= 1, a, amp[-1])
    g = 2 * a / T
    tail = (V - 1) * np.exp(-g)
    col = np.arange(N) % 4
    h = torch.zeros(N, D, dtype=torch.bfloat16)
    h[torch.arange(N), torch.from_numpy(col)] = torch.from_numpy(a).to(torch.bfloat16)
    assert (h.double().sum(1).numpy() == a).all()
    w = torch.zeros(V, D, dtype=torch.bfloat16, device=dev)
    w[:, :4] = -1
    for c, r in enumerate(first):
        w[r, c] = 1
    t = torch.tensor([first[c] for c in col], dtype=torch.int32)
    logp, lse, ent, ids, alt = (x.cpu().double().numpy() for x in pa.token_logprobs_forward(
        h.to(dev), w, t.to(dev), temperature=T, top=1))
    assert (ids[:, 0] == t.numpy()).all()
    u = 2.0 ** -24
    e_logp, e_ent = -np.log1p(tail), np.log1p(tail) + g * tail / (1 + tail)
    for got, want, bar, n in ((logp, e_logp, 40 * u * (1 + tail), "logp"), (alt[:, 0], e_logp, 40 * u * (1 + tail), "top_logp"),
                              (lse, a / T + np.log1p(tail), 40 * u * (1 + tail) + 4 * u * a / T, "lse"),
                              (ent, e_ent, u * (40 + 80 * (1 + g) * tail), "entropy")):
        err = np.abs(got - want)
        print(f"{n}: max err {err.max():.2e}, {(err / bar).max():.2f} of its bar")
        assert (err <= bar).all(), n


# one token to many: columns shared by four, two and no warps, CTA pairs; splits of
# 100 to 1,000 chunks of 32 columns
@pytest.mark.parametrize("N,V", [(1, 4_000_000), (60, 2_000_000), (100, 1_000_000), (1500, 400_000), (8192, 151_936)])
@pytest.mark.parametrize("T", [1.0, 0.5])
def test_a_likely_tokens_tail_is_summed(N, V, T, cuda_dev):
    """Thousands of tokens of 1e-9 each behind a likely one, whose probability
    alone is nearly 1: what they add in all is not rounded away chunk by chunk."""
    check_dominant(N, V, T, cuda_dev)


def test_infinities_and_nan_stay_in_their_rows(cuda_dev):
    N, V, D = 6, 300, 64
    H, W, t = inputs(N, V, D, 9)
    H[:, 0] = 1
    clean = run(H, W, t, cuda_dev, 1.0, 4)
    H2 = H.copy()
    H2[2, 5] = np.nan
    got = run(H2, W, t, cuda_dev, 1.0, 4)
    others = [0, 1, 3, 4, 5]
    for g, c in zip(got, clean):
        assert (g[others] == c[others]).all()
    assert np.isnan(got[1][2]) and np.isnan(got[2][2]) and (got[3][2] == -1).all() and (got[4][2] == -np.inf).all()
    # logits of -inf: no alternatives, nothing to the sums; a scored one has logp -inf
    W2 = np.zeros_like(W)
    W2[:, 1] = W[:, 1]
    W2[10:, 0] = -np.inf
    H3 = np.zeros_like(H)
    H3[:, :2] = np.abs(H[:, :2]) + 1 / 8
    H3[:, 2:] = 0
    # columns of zeros times -inf rows would be NaN: only column 0 is infinite there
    t3 = np.array([0, 1, 9, 10, 299, -1], np.int32)
    got = run(H3, W2, t3, cuda_dev, 1.0, 16)
    want = logprobs.forward(H3, W2[:10], np.where(t3 < 10, t3, -1), 1.0, 10)
    assert (got[3][:, :10] == want[3]).all() and (got[3][:, 10:] == -1).all() and (got[4][:, 10:] == -np.inf).all()
    assert np.abs(got[1] - want[1]).max() < 1e-5 and np.abs(got[2] - want[2]).max() < 1e-5
    assert (got[0][[3, 4]] == -np.inf).all() and got[0][5] == 0


@pytest.mark.parametrize("N", [1, 40, 100, 300])
@pytest.mark.parametrize("low,T", [(-1e38, 1.0), (-1e38, 0.7), (-3.3e38, 1.0), (-3.3e38, 2.0), (-1e34, 2.0), (-3e34, 1.0),
                                   (-1e12, 0.5), (-5e9, 1.0)])
def test_rows_masked_by_the_types_lowest_values(N, low, T, cuda_dev):
    """Vocabulary rows taken out by a bias of about the lowest bf16 value: whole
    chunks, tiles and splits of nothing but such logits, the first ones among
    them, count for nothing, whichever way low log2(e) / T rounds. (Their own logits differ by less than fp32 holds
    there, so only the other rows are asked for as alternatives.)"""
    V, D, top = 20_000, 64, 8
    H, W, t = inputs(N, V, D, 23)
    H[:, 0], W[:, 0] = 1, 0
    low = float(torch.tensor(low, dtype=torch.bfloat16))
    keep = np.r_[300:340, 9000:9005, 9100, 15_000:15_032, V - 3]
    masked = np.setdiff1d(np.arange(V), keep)
    t = keep[t % len(keep)].astype(np.int32)
    t[-1] = -1
    e_logp, e_lse, e_ent, e_ids, e_alt = logprobs.forward(H, W[keep], np.where(t < 0, -1, np.searchsorted(keep, t)), T, top)
    z = np.abs(H @ W[keep].T).max() / T
    W[masked, 0] = low
    got = run(H, W, t, cuda_dev, T, top)
    check(got, [e_logp, e_lse, e_ent, keep[e_ids], e_alt], V, z)
    # and their gradients are zero
    h, w, tt = dev_bf16(H, cuda_dev), dev_bf16(W, cuda_dev), torch.from_numpy(t).to(cuda_dev)
    _, lse, ent, _, _ = pa.token_logprobs_forward(h, w, tt, temperature=T)
    g = torch.from_numpy(synth.normals(3, 65, N).astype(np.float32)).to(cuda_dev)
    dh, dw = pa.token_logprobs_backward(h, w, tt, lse, ent, g, 0.3 * g, temperature=T)
    dh, dw = dh.double().cpu().numpy(), dw.double().cpu().numpy()
    assert np.isfinite(dh).all() and (dw[masked] == 0).all()
    eh, ew = logprobs.backward(H, W[keep], np.where(t < 0, -1, np.searchsorted(keep, t)), g.double().cpu().numpy(),
                               (0.3 * g).double().cpu().numpy(), T)
    assert np.linalg.norm(dw[keep] - ew) <= 2.0 ** -8 * np.linalg.norm(ew)
    assert np.linalg.norm(dh[:, 1:] - eh[:, 1:]) <= 2.0 ** -8 * np.linalg.norm(eh[:, 1:])



@pytest.mark.parametrize("N", [1, 40, 100, 300])
@pytest.mark.parametrize("low,T", [(-1e38, 1.0), (-1e38, 0.7), (-3.3e38, 2.0), (3e34, 1.0), (-5e9, 0.5), (0.0, 1e-20)])
def test_tokens_with_nothing_but_masked_logits(N, low, T, cuda_dev):
    """Logits that are all the same, however large: the softmax is uniform and
    lse is the logit itself as far as fp32 holds it. The last: a temperature so
    small that only the largest logits count, 100 equal ones of 199/64 in rows
    1, 201, ...; the target's is 1, and exact like the others."""
    V, D, top = 20_000, 64, 8
    H, W = np.zeros((N, D)), np.zeros((V, D))
    H[:, 0] = 1
    low = float(torch.tensor(low, dtype=torch.bfloat16))
    W[:, 0] = low
    t = (np.arange(N) * 41 % V).astype(np.int32)
    if low == 0:
        W[:, 0], t[:] = (-np.arange(V) % 200) / 64, 7
        W[7, 0] = 1
    logp, lse, ent, ids, alt = run(H, W, t, cuda_dev, T, top)
    bar = 2.0 ** -24 * (V / 32 + 32)
    if low == 0:
        assert np.abs(logp.astype(np.float64) * T * 64 / (64 - 199) - 1).max() <= 2.0 ** -22
        assert np.abs(ent - math.log(100)).max() <= bar and np.abs(alt + math.log(100)).max() <= bar
        assert (ids == 1 + 200 * np.arange(top)).all() and np.abs(lse.astype(np.float64) * T * 64 / 199 - 1).max() <= 2.0 ** -22
    else:
        assert np.abs(logp + math.log(V)).max() <= bar and np.abs(ent - math.log(V)).max() <= 12 * bar
        assert (ids == np.arange(top)).all() and np.abs(alt + math.log(V)).max() <= bar
        assert np.abs(lse / (low / T) - 1).max() <= 2.0 ** -22


@pytest.mark.parametrize("N,top", [(2, 5), (2, 20), (150, 8), (150, 32)])
def test_nan_rows_of_the_head_are_no_alternatives(N, top, cuda_dev):
    """A head row of NaN spoils every token's sums, but the alternatives are the
    other rows', in their order; whole groups of NaN rows among the first."""
    V, D = 4000, 64
    H, W, t = inputs(N, V, D, 19 + top)
    W2 = W.copy()
    dead = np.r_[0:40, 64:72, 133, 200:260, V - 1]
    W2[dead] = np.nan
    got = run(H, W2, t, cuda_dev, 1.0, top)
    alive = np.setdiff1d(np.arange(V), dead)
    order = alive[np.argsort(-(H @ W[alive].T), axis=1, kind="stable")[:, :top]]
    assert (got[3] == order).all()
    assert np.isnan(got[1]).all() and np.isnan(got[2]).all()


def test_the_same_bits_again_and_in_a_graph(cuda_dev):
    """Two calls, a call on another stream, and a captured call replayed on
    new inputs give the same bits; two graphs keep workspaces of their own."""
    N, V, D, top = 70, 4000, 256, 8
    sets = [[dev_bf16(x, cuda_dev) for x in inputs(N, V, D, s)[:2]] + [torch.from_numpy(inputs(N, V, D, s)[2]).to(cuda_dev)]
            for s in (1, 2)]
    want = [pa.token_logprobs_forward(*s, top=top) for s in sets]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        again = pa.token_logprobs_forward(*sets[0], top=top)
    side.synchronize()
    for a, b in zip(again, want[0]):
        assert torch.equal(a, b)
    static = [x.clone() for x in sets[0]]
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = pa.token_logprobs_forward(*static, top=top)
        graphs.append((g, out))
    for s, w in ((1, want[1]), (0, want[0])):
        for x, y in zip(static, sets[s]):
            x.copy_(y)
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        for _, out in graphs:
            for a, b in zip(out, w):
                assert torch.equal(a, b)


def test_one_token_is_a_row_of_many(cuda_dev):
    """A token scored alone gives what it gives in a batch, within the bars."""
    N, V, D = 200, 9001, 128
    H, W, t = inputs(N, V, D, 12)
    want = logprobs.forward(H, W, t, 1.0, 5)
    for i in (0, 1, 199):
        check(run(H[i:i + 1], W, t[i:i + 1], cuda_dev, 1.0, 5), [x[i:i + 1] for x in want], V, np.abs(H @ W.T).max())


# ------------------------------------------------------------------ backward
# bf16 keeps 8 significant bits: in [1, 2) its step is 2^-7, so a rounding is off
# by at most half of that, 2^-8 of the value. dz is rounded to bf16 and the
# gradient to bf16 again; the fp32 sums between are far more exact. So an
# element of the gradient is within 2^-8 sum |dz||w| + 2^-8 |gradient| of the
# exact one. Over a tensor the roundings have random signs and are spread
# evenly over the half steps (1 / sqrt(3) of the largest, and 1 / 1.4 for the
# mean place in [1, 2)): 1.6e-3 of the norm for each of the two, 2.3e-3
# together, so 2^-8 = 3.9e-3 is the bar for the norm.
BWD = [
    (1, 33, 64, True, True, 1.0), (2, 1, 64, True, True, 1.0), (5, 1000, 128, True, True, 0.7),
    (130, 1003, 192, True, True, 1.3), (300, 5000, 256, True, False, 1.0), (300, 5000, 256, False, True, 1.0),
    (96, 32003, 128, True, True, 1.0), (4500, 17000, 64, True, True, 1.0), (257, 130, 1088, True, True, 2.0),
    # a last chunk of 100 vocabulary rows, fewer than dH's contraction has runs
    (3000, 22372, 64, False, True, 1.0),
]


def bwd(H, W, t, g, e, dev, T, head):
    h, w, tt = dev_bf16(H, dev), dev_bf16(W, dev), torch.from_numpy(t).to(dev)
    _, lse, ent, _, _ = pa.token_logprobs_forward(h, w, tt, temperature=T)
    f = lambda x: None if x is None else torch.from_numpy(x.astype(np.float32)).to(dev)
    ws = torch.empty(pa.pa_logp_bwd_workspace_bytes(h.shape[0], w.shape[0], h.shape[1]), dtype=torch.uint8, device=dev)
    got = pa.token_logprobs_backward(h, w, tt, lse, ent, f(g), f(e), temperature=T, train_head=head, ws=ws)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    return [None if x is None else x.float().cpu().numpy().astype(np.float64) for x in got]


def upstream(N, t, V, seed, entropy):
    g = synth.normals(seed, 63, N).astype(np.float32).astype(np.float64)
    e = 0.5 * synth.normals(seed, 64, N).astype(np.float32).astype(np.float64) if entropy else None
    return g, None if e is None else e.astype(np.float32).astype(np.float64)


def check_grads(got, H, W, t, g, e, T, dz_step=2.0 ** -8):
    N, V = H.shape[0], W.shape[0]
    z = H @ W.T / T
    lp = z - z.max(1, keepdims=True)
    lp -= np.log(np.exp(lp).sum(1, keepdims=True))
    p = np.exp(lp)
    gs = np.where((t >= 0) & (t < V), g, 0)
    dz = -gs[:, None] * p
    ok = gs != 0
    dz[np.arange(N)[ok], t[ok]] += gs[ok]
    # what dz is made of before its terms cancel bounds its own error (2e-5 of it)
    size = np.abs(gs)[:, None] * p
    size[np.arange(N)[ok], t[ok]] += np.abs(gs[ok])
    if e is not None:
        ent = -(p * lp).sum(1, keepdims=True)
        dz -= e[:, None] * p * (lp + ent)
        size += np.abs(e)[:, None] * p * (np.abs(lp) + ent)
    dz, size = dz / T, size / T
    for x, a, b, s, n in ((got[0], dz, W, size, "dH"), (got[1], dz.T, H, size.T, "dW")):
        if x is None:
            continue
        exact = a @ b
        norm = np.linalg.norm(exact)
        rel = np.linalg.norm(x - exact) / norm if norm else np.abs(x).max()
        bound = dz_step * (np.abs(a) @ np.abs(b)) + 2e-5 * (s @ np.abs(b)) + 2.0 ** -8 * np.abs(exact)
        worst = (np.abs(x - exact) / np.maximum(bound, 1e-30)).max()
        print(f"{n}: relL2 {rel:.2e}, worst element {worst:.2f} of its bound")
        assert worst <= 1.01, n
        if x.size > 1000:
            assert rel <= 2.0 ** -8, n


@pytest.mark.parametrize("N,V,D,head,entropy,T", BWD)
def test_backward_matches_the_formula(N, V, D, head, entropy, T, cuda_dev):
    H, W, t = inputs(N, V, D, 3 * N + V)
    g, e = upstream(N, t, V, N, entropy)
    if N > 6:
        g[5], t[6] = 0, -1
        if e is not None:
            e[5] = e[6] = 0
    got = bwd(H, W, t, g, e, cuda_dev, T, head)
    assert (got[1] is None) == (not head)
    check_grads(got, H, W, t, g, e, T)
    if N > 6:
        assert (got[0][5] == 0).all() and (got[0][6] == 0).all()  # no gradient, exactly


# Up to 128 tokens dz is kept as two bf16 terms: the second rounds what the first
# leaves (2^-8 of the value at most), so 2^-16 of the value is lost. A single
# token's gradient is then as good as its own rounding, whatever the one large
# value's rounding at its target would have been.
@pytest.mark.parametrize("N,V,D,head", [(1, 1003, 64, True), (1, 8203, 320, False), (2, 17125, 192, True), (63, 700, 1088, True),
                                        (65, 3000, 512, True), (96, 5000, 128, False), (128, 4099, 320, True),
                                        (128, 270001, 64, True)])  # two chunks of the vocabulary
@pytest.mark.parametrize("T", [1.0, 0.7])
def test_gradients_of_few_tokens_are_exact_but_for_their_own_rounding(N, V, D, head, T, cuda_dev):
    H, W, t = inputs(N, V, D, 7 * N + V)
    g, e = upstream(N, t, V, N + 1, True)
    check_grads(bwd(H, W, t, g, e, cuda_dev, T, head), H, W, t, g, e, T, dz_step=2.0 ** -16)


@pytest.mark.parametrize("N,head", [(3, True), (3, False), (70, True)])
def test_few_tokens_over_a_vocabulary_of_two_chunks(N, head, cuda_dev):
    """The transposed dz, padded to 64 tokens a row, bounds the chunk: 2^20 rows
    for 3 tokens and 2^19 for 70."""
    V, D = (1 << 20 if N <= 64 else 1 << 19) + 1003, 64
    H, W, t = inputs(N, V, D, N)
    t[0], t[2] = V - 1, V - 1003
    g, e = upstream(N, t, V, N, True)
    check_grads(bwd(H, W, t, g, e, cuda_dev, 1.0, head), H, W, t, g, e, 1.0, dz_step=2.0 ** -16)


@pytest.mark.parametrize("N", [5, 300])
def test_the_widest_hidden_size(N, cuda_dev):
    """D = 16,384, both directions."""
    V, D = 1003, 16384
    H, W, t = inputs(N, V, D, 41)
    check(run(H, W, t, cuda_dev, 1.0, 8), logprobs.forward(H, W, t, 1.0, 8), V, np.abs(H @ W.T).max())
    g, e = upstream(N, t, V, 41, True)
    check_grads(bwd(H, W, t, g, e, cuda_dev, 1.0, True), H, W, t, g, e, 1.0, dz_step=2.0 ** -16 if N <= 128 else 2.0 ** -8)


@pytest.mark.parametrize("T", [1e-3, 30.0, 1e30, 3e38])
def test_temperatures_far_from_one(T, cuda_dev):
    """Nearly greedy to uniform; the gradient's 1 / T with it (where 1 / T is a
    number that bf16 holds to eight bits)."""
    N, V, D = 9, 3000, 64
    H, W, t = inputs(N, V, D, 43)
    check(run(H, W, t, cuda_dev, T, 4), logprobs.forward(H, W, t, T, 4), V, np.abs(H @ W.T).max() / T)
    if T <= 1e30:
        g, e = upstream(N, t, V, 43, True)
        dh, dw = bwd(H, W, t, g, e, cuda_dev, T, True)
        eh, ew = logprobs.backward(H, W, t, g, e, T)
        assert np.linalg.norm(dw - ew) <= 2.0 ** -8 * np.linalg.norm(ew)
        # a token's row: p is off by 2^-24 (3 * 1.45 Z) of itself through z and lse, and
        # at T = 1e-3, Z is some thousands: 1e-3 of what dz is made of before it cancels
        Z = np.abs(H @ W.T).max() / T
        size = np.linalg.norm(np.abs(g)[:, None] / T * np.abs(W).max(0), axis=1) * 2 + np.linalg.norm(eh, axis=1)
        bar = 2.0 ** -8 * np.linalg.norm(eh, axis=1) + 2.0 ** -24 * (8 * Z + 64) * size * (1 + np.abs(e) * Z)
        assert (np.linalg.norm(dh - eh, axis=1) <= bar).all()


@pytest.mark.parametrize("N", [9, 100, 300])
@pytest.mark.parametrize("low", [-5e9, -1e12, 5e9, -1e34, -3e34, -1e38, 3e34])
def test_a_token_whose_lse_fp32_cannot_hold_spoils_no_other(N, low, cuda_dev):
    """Tokens whose logits are all of about `low`: lse rounds to that, and what
    p = exp(z - lse) is, fp32 cannot tell; but it is not above 1, so the gradients
    stay finite (but for column 0 of the tokens themselves, which sums 3,000 dz of
    order 1 times `low`: 1e38 and more), and the other tokens' are what they are
    without."""
    V, D = 3000, 64
    H, W, t = inputs(N, V, D, 47)
    t = np.where(t < 0, 3, t % V).astype(np.int32)
    H[:, 0], W[:, 0] = 0, float(torch.tensor(low, dtype=torch.bfloat16))
    bad = np.arange(N) % 7 == 2
    H[bad, 0] = 1
    g, e = upstream(N, t, V, 47, True)
    dh, dw = bwd(H, W, t, g, e, cuda_dev, 1.0, True)
    assert np.isfinite(dh[:, 1:]).all() and np.isfinite(dh[~bad]).all() and np.isfinite(dw).all()
    # columns 1 on of the others' rows (their column 0 sums dz times the huge column,
    # where dz is 0 in all but its rounding)
    eh, _ = logprobs.backward(H[~bad], W, t[~bad], g[~bad], e[~bad], 1.0)
    assert np.linalg.norm((dh[~bad] - eh)[:, 1:]) <= 2.0 ** -8 * np.linalg.norm(eh[:, 1:])


@pytest.mark.parametrize("N", [9, 300])
def test_a_nan_state_shows_in_its_gradient_alone(N, cuda_dev):
    V, D = 3000, 64
    H, W, t = inputs(N, V, D, 53)
    g, e = upstream(N, t, V, 53, True)
    want, _ = bwd(H, W, t, g, e, cuda_dev, 1.0, True)
    H2 = H.copy()
    H2[4, 7] = np.nan
    got, dw = bwd(H2, W, t, g, e, cuda_dev, 1.0, True)
    others = np.arange(N) != 4
    assert np.isnan(got[4]).all() and np.isnan(dw).all() and (got[others] == want[others]).all()


def test_backward_matches_the_oracle_and_differences(cuda_dev):
    """Against the oracle's gradient, and the change of the loss along it:
    for a step s along the direction of the gradient itself the loss changes by
    s |dH|^2 up to third order (1e-3 of it at this step)."""
    N, V, D, T = 9, 64, 64, 0.8
    H, W, t = inputs(N, V, D, 31)
    g, e = upstream(N, t, V, 31, True)
    dh, dw = bwd(H, W, t, g, e, cuda_dev, T, True)
    eh, ew = logprobs.backward(H, W, t, g, e, T)
    assert np.linalg.norm(dh - eh) <= 2.0 ** -8 * np.linalg.norm(eh)
    assert np.linalg.norm(dw - ew) <= 2.0 ** -8 * np.linalg.norm(ew)

    def loss(H, W):
        logp, _, ent, _, _ = logprobs.forward(H, W, t, T)
        return (g * logp + e * ent).sum()
    for d, f in ((dh, lambda s: loss(H + s * dh, W)), (dw, lambda s: loss(H, W + s * dw))):
        s = 1e-3 / np.linalg.norm(d)
        slope = (f(s) - f(-s)) / (2 * s)
        assert abs(slope / (d * d).sum() - 1) < 2.0 ** -7 + 1e-3


def test_backward_frozen_head_bits_and_graph(cuda_dev):
    """Without the head's gradient dhidden has the same bits; so does a second
    call and a captured one replayed beside an eager one."""
    N, V, D = 200, 9000, 128
    H, W, t = inputs(N, V, D, 15)
    h, w, tt = dev_bf16(H, cuda_dev), dev_bf16(W, cuda_dev), torch.from_numpy(t).to(cuda_dev)
    _, lse, ent, _, _ = pa.token_logprobs_forward(h, w, tt)
    g, e = (torch.from_numpy(x.astype(np.float32)).to(cuda_dev) for x in upstream(N, t, V, 4, True))
    dh, dw = pa.token_logprobs_backward(h, w, tt, lse, ent, g, e)
    dh2, none = pa.token_logprobs_backward(h, w, tt, lse, ent, g, e, train_head=False)
    assert none is None and torch.equal(dh, dh2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gw = pa.token_logprobs_backward(h, w, tt, lse, ent, g, e)
    for _ in range(2):
        gh.zero_()
        gw.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gh, dh) and torch.equal(gw, dw)


@pytest.mark.parametrize("N", [1, 100])
def test_few_tokens_bits_graph_and_two_streams(N, cuda_dev):
    """The head's and the states' gradients of few tokens run side by side: the
    same bits again, replayed, and in two calls at once on streams of their own."""
    V, D = 20011, 576
    H, W, t = inputs(N, V, D, 16)
    h, w, tt = dev_bf16(H, cuda_dev), dev_bf16(W, cuda_dev), torch.from_numpy(t).to(cuda_dev)
    _, lse, ent, _, _ = pa.token_logprobs_forward(h, w, tt)
    g, e = (torch.from_numpy(x.astype(np.float32)).to(cuda_dev) for x in upstream(N, t, V, 4, True))
    dh, dw = pa.token_logprobs_backward(h, w, tt, lse, ent, g, e)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gh, gw = pa.token_logprobs_backward(h, w, tt, lse, ent, g, e)
    for _ in range(2):
        gh.zero_()
        gw.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gh, dh) and torch.equal(gw, dw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    made = [[], []]
    for _ in range(4):
        for s, m in zip(streams, made):
            with torch.cuda.stream(s):
                m.append(pa.token_logprobs_backward(h, w, tt, lse, ent, g, e))
    torch.cuda.synchronize()
    for m in made:
        for x, y in m:
            assert torch.equal(x, dh) and torch.equal(y, dw)


def test_the_mean_nll_is_the_cross_entropys(cuda_dev):
    """At temperature 1 logp is minus the cross-entropy's NLL, and its gradient
    the cross-entropy's with the sign turned."""
    N, V, D = 150, 2000, 128
    H, W, t = inputs(N, V, D, 21)
    h, w, tt = dev_bf16(H, cuda_dev), dev_bf16(W, cuda_dev), torch.from_numpy(t).to(cuda_dev)
    nll, lse_x, _ = pa.linear_cross_entropy_forward(h, w, tt)
    logp, lse, ent, _, _ = pa.token_logprobs_forward(h, w, tt)
    assert (logp + nll).abs().max() < 2e-5 and (lse - lse_x).abs().max() < 2e-5
    g = torch.full((N,), 1.0 / N, device=cuda_dev)
    a = pa.linear_cross_entropy_backward(h, w, tt, lse_x, g)
    b = pa.token_logprobs_backward(h, w, tt, lse, ent, -g)
    for x, y in zip(a, b):
        # each is within 2^-8 of the exact gradient
        assert (x.float() - y.float()).norm() <= 2.0 ** -7 * x.float().norm()


def test_a_head_past_32_bit_offsets(cuda_dev):
    """V * D beyond 2^31 elements, both directions, against fp64 on the device.
    (The backward's tokens sit in one tile, its vocabulary in one chunk.)"""
    N, V, D, top = 3, 540_001, 4096, 8
    g = torch.Generator(device=cuda_dev).manual_seed(1)
    w = torch.empty(V, D, dtype=torch.bfloat16, device=cuda_dev)
    for a in range(0, V, 60_000):
        n = min(60_000, V - a)
        w[a:a + n] = torch.randint(-15, 16, (n, D), generator=g, device=cuda_dev).float() / 256
    h = (torch.randint(-15, 16, (N, D), generator=g, device=cuda_dev).float() / 8).bfloat16()
    t = torch.tensor([V - 1, 5, 500_000], dtype=torch.int32, device=cuda_dev)
    logp, lse, ent, ids, alt = pa.token_logprobs_forward(h, w, t, top=top)
    z = torch.cat([h.double() @ w[a:a + 60_000].double().T for a in range(0, V, 60_000)], 1)
    lp = torch.log_softmax(z, 1)
    want = [lp[torch.arange(N), t.long()], torch.logsumexp(z, 1), -(lp.exp() * lp).sum(1), torch.sort(z, dim=1, descending=True, stable=True).indices[:, :top]]
    # the bars of check(): V / 32 chunk sums are spread over the splits here
    u = 2.0 ** -24
    bar = 3 * 1.45 * z.abs().max().item() * u + 4 * u + u * (V / 32 / 100 + 32) + 8 * u * z.abs().max().item()
    assert (logp.double() - want[0]).abs().max() <= bar and (lse.double() - want[1]).abs().max() <= bar
    assert (ent.double() - want[2]).abs().max() <= bar * (2 + want[2].max() + math.log(V) + 1)
    assert torch.equal(ids.long(), want[3])
    gl = torch.tensor([1.0, -2.0, 0.5], device=cuda_dev)
    dh, dw = pa.token_logprobs_backward(h, w, t, lse, ent, gl, 0.1 * gl)
    dz = -lp.exp() * (gl.double()[:, None] + 0.1 * gl.double()[:, None] * (lp + want[2][:, None]))
    dz[torch.arange(N), t.long()] += gl.double()
    for a, b in ((0, 2000), (499_000, 501_000), (V - 2000, V)):
        exact = dz[:, a:b].T @ h.double()
        assert (dw[a:b].double() - exact).norm() <= 2.0 ** -8 * exact.norm()
    exact = sum(dz[:, a:a + 60_000] @ w[a:a + 60_000].double() for a in range(0, V, 60_000))
    assert (dh.double() - exact).norm() <= 2.0 ** -8 * exact.norm()


def test_tokens_past_32_bit_offsets(cuda_dev):
    """A chunk's dz and its transposed copy beyond 2^31 elements (8.6 million tokens
    by 256 vocabulary rows, two chunks), against fp64 on the device."""
    N, V, D, top = 8_600_003, 300, 64, 2
    gen = torch.Generator(device=cuda_dev).manual_seed(2)
    h = (torch.randint(-15, 16, (N, D), generator=gen, device=cuda_dev, dtype=torch.int8).bfloat16() / 8)
    w = (torch.randint(-15, 16, (V, D), generator=gen, device=cuda_dev).float() / 32).bfloat16()
    t = torch.randint(-1, V, (N,), generator=gen, device=cuda_dev, dtype=torch.int32)
    g = torch.randn(N, generator=gen, device=cuda_dev)
    e = 0.5 * torch.randn(N, generator=gen, device=cuda_dev)
    logp, lse, ent, ids, alt = pa.token_logprobs_forward(h, w, t, top=top)
    ws = torch.empty(pa.pa_logp_bwd_workspace_bytes(N, V, D), dtype=torch.uint8, device=cuda_dev)
    dh, dw = pa.token_logprobs_backward(h, w, t, lse, ent, g, e, ws=ws)
    torch.cuda.synchronize()
    assert pa.pa_device_status(ws) == 0
    del ws
    u, wd = 2.0 ** -24, w.double()
    exact_w, err_h, norm_h = torch.zeros(V, D, dtype=torch.float64, device=cuda_dev), 0.0, 0.0
    for a in range(0, N, 400_000):
        s = slice(a, min(N, a + 400_000))
        hd, ti = h[s].double(), t[s].long()
        raw = hd @ wd.T
        lp = torch.log_softmax(raw, 1)
        en = -(lp.exp() * lp).sum(1)
        scored = ti >= 0
        want = torch.where(scored, lp.gather(1, ti.clamp(min=0)[:, None])[:, 0], 0.0)
        Z = raw.abs().max().item()
        bar = 3 * 1.45 * Z * u + 4 * u + u * (V / 32 + 32) + 8 * u * (Z + math.log(V))
        assert (logp[s].double() - want).abs().max() <= bar
        assert (lse[s].double() - torch.logsumexp(raw, 1)).abs().max() <= bar
        assert (ent[s].double() - en).abs().max() <= bar * (3 + 2 * math.log(V))
        assert torch.equal(ids[s].long(), torch.sort(raw, dim=1, descending=True, stable=True).indices[:, :top])
        gs = torch.where(scored, g[s], 0.0).double()
        dz = -lp.exp() * (gs[:, None] + e[s].double()[:, None] * (lp + en[:, None]))
        dz.scatter_add_(1, ti.clamp(min=0)[:, None], gs[:, None])
        x = dz @ wd
        err_h += (dh[s].double() - x).square().sum().item()
        norm_h += x.square().sum().item()
        exact_w += dz.T @ hd
    assert err_h ** 0.5 <= 2.0 ** -8 * norm_h ** 0.5
    assert (dw.double() - exact_w).norm() <= 2.0 ** -8 * exact_w.norm()


def test_refused_shapes_and_devices(cuda_dev):
    h, w = torch.zeros(4, 64, dtype=torch.bfloat16, device=cuda_dev), torch.zeros(9, 64, dtype=torch.bfloat16, device=cuda_dev)
    t = torch.zeros(4, dtype=torch.int32, device=cuda_dev)
    with pytest.raises(ValueError):
        pa.token_logprobs_forward(h.float(), w, t)
    with pytest.raises(ValueError):
        pa.token_logprobs_forward(h, w, t.long())
    with pytest.raises(ValueError):
        pa.token_logprobs_forward(h, w.cpu(), t)
    with pytest.raises(ValueError):
        pa.token_logprobs_forward(h.t().contiguous().t(), w, t)
    with pytest.raises(pa.PAError):
        pa.token_logprobs_forward(h, w, t, temperature=0.0)
    with pytest.raises(pa.PAError):
        pa.token_logprobs_forward(h, w, t, ws=torch.empty(64, dtype=torch.uint8, device=cuda_dev))
