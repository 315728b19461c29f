"""The paged cache and the attention over it on the GPU against the fp64 oracle.

Attention: with A = sum_j w_j |v_j|, the weights' rounding to bf16 (2^-8 of each) moves an
output by at most 2^-8 A through the product and, where the normaliser sums the
rounded weights, by 2^-8 A once more; the result's own rounding is 2^-8 |out|. Scores: the
products of bf16 numbers are exact and each of D / 16 additions to an fp32 sum loses at
most 2^-23 of what has come together, at most Z = max sum_c |q_c k_c| scale; the scale in
base 2 rounds twice. So a score is within (D / 16 + 2) 2^-23 Z <= 10 * 2^-23 Z of itself,
a weight within twice that, the exponential 2^-22. lse adds what a sum of n terms in
fp32 loses, at most (64 + n / 64) 2^-24.

What the cache holds outside the sequences' tokens is NaN throughout."""
import math

import numpy as np
import pytest
import torch

import oracle
import segment_masked_causal_gb300 as pa
import synth
from oracle import paged, rotary

pytestmark = pytest.mark.gpu
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    from segment_masked_causal_gb300 import build
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


class Step:
    """Sequences of (new, total) tokens over a cache of shuffled pages."""

    def __init__(self, lens, Hq, Hkv, D, page, dev, seed=1, order="phnd", tail=0, spare=2, width=None, dtype=torch.bfloat16):
        self.rng = rng = np.random.default_rng(seed)
        self.lens, self.Hq, self.Hkv, self.D, self.page, self.dev = lens, Hq, Hkv, D, page, dev
        self.start = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32)
        self.kv = np.array([t for _, t in lens], np.int32)
        self.T = int(self.start[-1]) + tail
        need = [-(-t // page) for _, t in lens]
        pages = sum(need) + spare
        perm = rng.permutation(pages)
        self.table = np.full((len(lens), width or max(max(need), 1) + 1), pages + 5, np.int32)  # what is not used is no page
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = perm[at:at + n][:self.table.shape[1]]
            at += n
        g = torch.Generator(device=dev).manual_seed(seed)
        shape = (pages, Hkv, page, D) if order == "phnd" else (pages, page, Hkv, D)
        self.kp, self.vp = (torch.full(shape, NAN, device=dev, dtype=dtype) for _ in range(2))
        if order != "phnd":
            self.kp, self.vp = self.kp.transpose(1, 2), self.vp.transpose(1, 2)
        for x in (self.kp, self.vp):
            for s, (_, t) in enumerate(lens):
                for j in range(0, min(t, page * self.table.shape[1]), page):
                    n = min(page, t - j)
                    x[int(self.table[s, j // page]), :, :n] = torch.randn(Hkv, n, D, generator=g, device=dev).to(dtype)
        self.q = torch.randn(max(self.T, 1), Hq, D, generator=g, device=dev).to(dtype)[:self.T]
        self.cache = pa.PagedCache(self.kp, self.vp)
        self.upload()

    def upload(self):
        self.d = [torch.from_numpy(x).to(self.dev) for x in (self.table, self.start, self.kv)]

    def forward(self, **kw):
        out = torch.full_like(self.q, 7.0)
        lse = torch.full((self.T, self.Hq), 7.0, device=self.dev)
        ws = pa.paged_workspace(self.q, self.cache)
        pa.paged_forward(self.q, self.cache, *self.d, out=out, lse=lse, ws=ws, **kw)
        torch.cuda.synchronize()
        assert pa.pa_device_status(ws) == 0
        return out, lse

    def check(self, out, lse, scale=None):
        want, wl, A, Z = paged.attention(f64(self.q), f64(self.kp), f64(self.vp), self.table, self.start, self.kv, scale)
        got, gl = f64(out), f64(lse)
        mine = ~np.isnan(wl)
        assert (got[~mine] == 7).all() and (gl[~mine] == 7).all()  # nobody's rows
        got, gl, want, wl, A, Z = got[mine], gl[mine], want[mine], wl[mine], A[mine], Z[mine]
        n = max(t for _, t in self.lens)
        score = 10 * 2.0 ** -23 * Z
        tol = (2 * 2.0 ** -8 + 2.0 ** -12 + 2 * score[..., None]) * A + 2.0 ** -8 * np.abs(want)
        assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) - tol).max()
        none = np.isneginf(wl)
        assert (gl[none] == -np.inf).all() and (got[none] == 0).all()
        err = np.abs(gl[~none] - wl[~none])
        assert (err <= score[~none] + 2.0 ** -22 + (64 + n / 64) * 2.0 ** -24 + 2.0 ** -23 * np.abs(wl[~none])).all(), err.max()


HEADS = [(1, 1), (4, 1), (8, 2), (7, 1), (10, 2), (6, 6), (48, 3)]


@pytest.mark.parametrize("D", [64, 96, 128])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("lens", [
    [(1, 1)], [(1, 15), (1, 16), (1, 17), (1, 129), (1, 128), (1, 127)], [(5, 5), (3, 200), (1, 400), (9, 9)],
    [(0, 0), (1, 33), (0, 70), (40, 100), (0, 0)], [(130, 300), (64, 64)]], ids=["first", "one", "few", "none", "chunk"])
def test_lengths_and_pages(cuda_dev, D, page, lens):
    s = Step(lens, 8, 2, D, page, cuda_dev, seed=D + page)
    s.check(*s.forward())


@pytest.mark.parametrize("Hq,Hkv", HEADS + [(128, 1)])
@pytest.mark.parametrize("order", ["phnd", "pnhd"])
@pytest.mark.parametrize("D", [64, 128])
def test_heads_orders_and_rows_of_nobody(cuda_dev, Hq, Hkv, order, D):
    s = Step([(1, 300), (37, 150), (2, 2), (0, 9)], Hq, Hkv, D, 32, cuda_dev, seed=Hq, order=order, tail=11)
    s.check(*s.forward())


@pytest.mark.parametrize("lens", [[(1, 20000)], [(3, 9000), (1, 50), (200, 5000)], [(1, 3 * i + 1) for i in range(400)]],
                         ids=["long", "mixed", "many"])
@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 64), (5, 1, 96), (8, 2, 128)])
def test_long_and_many(cuda_dev, lens, Hq, Hkv, D):
    s = Step(lens, Hq, Hkv, D, 64, cuda_dev, seed=8)
    a, b = s.forward(), s.forward()
    s.check(*a)
    assert all(torch.equal(x, y) for x, y in zip(a, b))  # bit for bit


@pytest.mark.parametrize("visits", [6, 7, 8, 9])
@pytest.mark.parametrize("G,D", [(4, 96), (8, 128), (1, 64)])
def test_longest_context_without_a_cut(cuda_dev, visits, G, D):
    """Contexts that fill the page table's width, just below and above what an item needs to be
    cut: whole items leave no parts to be joined, longer ones do."""
    n = visits * 128
    s = Step([(1, n), (9, n), (140, n), (2, n - 1), (33, 70)], 2 * G, 2, D, 64, cuda_dev, seed=visits)
    s.table = np.ascontiguousarray(s.table[:, :n // 64])
    s.upload()
    a, b = s.forward(), s.forward()
    s.check(*a)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("G,D", [(2, 64), (4, 128)])
def test_items_of_every_kind_in_turn(cuda_dev, seed, G, D):
    """Short items that one softmax group takes alone, items that both share and pairs of
    tiles, one behind the other in every order: the groups meet where they have to."""
    rng = np.random.default_rng(seed)
    kinds = [(1, 60), (1, 130), (20, 100), (1, 300), (3, 90), (9, 520), (1, 700), (70, 260), (25, 400), (0, 0)]
    lens = [kinds[i] for i in rng.choice(len(kinds), 700, p=[.2, .1, .2, .1, .1, .05, .1, .02, .08, .05])]
    s = Step(lens, 2 * G, 2, D, 64, cuda_dev, seed=seed)
    a = s.forward()
    s.check(*a)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(a, s.forward()))


def test_many_sequences(cuda_dev):
    s = Step([((i * 7) % 3, (i * 7) % 3 + i % 40) for i in range(3000)], 2, 1, 64, 16, cuda_dev, seed=9, tail=3)
    s.check(*s.forward())


@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (3, 1), (8, 1), (10, 2), (64, 1)])
@pytest.mark.parametrize("D", [64, 96, 128])
def test_rows_of_a_tile(cuda_dev, Hq, Hkv, D):
    """New tokens around the borders at which a tile is held four times, alone, or with
    the next one: 8 and 128 rows, and what is left behind the last pair."""
    G = Hq // Hkv
    few, tile = max(1, 8 // G), 128 // G
    counts = sorted({1, 2, few, few + 1, tile - 1, tile, tile + 1, 2 * tile - 1, 2 * tile, 2 * tile + 1, 5 * tile + 3} - {0})
    s = Step([(n, n + 100 * (i % 3)) for i, n in enumerate(counts)], Hq, Hkv, D, 16, cuda_dev, seed=G + D)
    s.check(*s.forward())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [1, 3, 40, 100])
def test_items_cut_between_many(cuda_dev, D, new):
    """Few items over a long context: each is cut into many parts, of one tile and of two."""
    s = Step([(new, 12000 + new)], 4, 1, D, 128, cuda_dev, seed=D + new)
    s.check(*s.forward())


def test_costs_in_units_of_many_keys(cuda_dev):
    """Tables so wide that the costs of a step cannot be counted in keys in 32 bits."""
    s = Step([(1, 700), (90, 300), (2, 5000)], 8, 2, 64, 256, cuda_dev, seed=14, width=1 << 22)
    s.check(*s.forward())


@pytest.mark.parametrize("scale", [0.02, 1.0])
def test_scale_and_large_scores(cuda_dev, scale):
    s = Step([(4, 500), (1, 77)], 4, 2, 128, 16, cuda_dev, seed=10)
    s.q.mul_(4)
    s.check(*s.forward(scale=scale), scale=scale)


@pytest.mark.parametrize("page", [16, 128])
def test_pages_that_are_not_there(cuda_dev, page):
    """Page numbers outside the cache at the start, in the middle and at the end,
    a sequence longer than its row of the table, and rows that see nothing at all."""
    s = Step([(3, 1000), (20, 700), (1, 300), (4, 260), (2, 40)], 4, 2, 64, page, cuda_dev, seed=11)
    n = 1000 // page
    s.table[0, :n // 2] = -1
    s.table[1, 1] = s.kp.shape[0]
    s.table[1, 3:5] = 2 ** 31 - 1
    s.table[2, :] = -2 ** 31
    s.kv[3] = s.table.shape[1] * page + 50  # past the table
    s.table[3, :] = s.table[4, 0]           # one page again and again
    s.kv[4] = 1                             # two new tokens of a sequence of one: the first lies before its start
    s.kp[s.table[4, 0]], s.vp[s.table[4, 0]] = s.kp[s.table[0, n - 1]], s.vp[s.table[0, n - 1]]  # no NaN on it
    s.upload()
    s.check(*s.forward())


def test_arrays_out_of_range_are_taken_into_it(cuda_dev):
    """q_start and kv_len that describe no step: in bounds all the same, and the
    sequences that are described well come out right."""
    s = Step([(2, 50), (3, 60), (1, 70)], 4, 2, 64, 16, cuda_dev, seed=12)
    want, wl = s.forward()
    s.start[0] = -5  # as 0
    s.start[3] = 1000  # as T
    s.upload()
    out, lse = s.forward()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    s.kv[1] = -7  # as 0: three tokens that see nothing
    s.upload()
    out, lse = s.forward()
    assert torch.equal(out[:2], want[:2]) and (out[2:5] == 0).all() and (lse[2:5] == -math.inf).all()
    s.start[:] = [3, 1, 6, 2]  # falling
    s.upload()
    s.forward()
    r = pa.Rotary(64)
    x = torch.zeros(6, 2, 64, device=cuda_dev, dtype=torch.bfloat16)
    pa.paged_append(s.cache, None, x, x, *s.d, rotary=r)
    torch.cuda.synchronize()


def test_strided_rows(cuda_dev):
    s = Step([(3, 90), (20, 33)], 8, 2, 96, 16, cuda_dev, seed=13)
    want, wl = s.forward()
    wide = torch.full((s.T, 12, 104), NAN, device=cuda_dev, dtype=torch.bfloat16)
    wide[:, 2:10, :96] = s.q
    s.q = wide[:, 2:10, :96]
    outs = torch.full((8, s.T, 96), 7.0, device=cuda_dev, dtype=torch.bfloat16).transpose(0, 1)  # heads first
    lse = torch.empty(s.T, 8, device=cuda_dev)
    pa.paged_forward(s.q, s.cache, *s.d, out=outs, lse=lse)
    assert torch.equal(outs, want) and torch.equal(lse, wl)
    outs, lse = pa.paged_forward(s.q, s.cache, *s.d)
    assert torch.equal(outs, want) and outs.is_contiguous()


# ------------------------------------------------------------------ appending
def append_want(s, k, v, q, r, pos=None):
    """Cache and queries after the step, and the keys' and queries' tolerances."""
    kp, vp, out = f64(s.kp), f64(s.vp), None if q is None else f64(q)
    tk, tq = np.zeros_like(kp), None if q is None else np.zeros_like(out)
    K, V = f64(k), f64(v)

    def turn(x, at):
        if r is None:
            return x, np.zeros_like(x)
        y = rotary.rotate(x, np.array([at]), r.frequencies, r.amplitude, r.interleaved)
        return y, 2.0 ** -21 * rotary.weight(x, r.frequencies, r.interleaved) * r.amplitude + 2.0 ** -8 * np.abs(y)
    for t, seq, p, page, row in paged.places(s.start, s.kv, s.table, kp.shape[0], s.page):
        at = p if pos is None else int(pos[t])
        if page >= 0:
            kp[page, :, row], tk[page, :, row] = turn(K[t], at)
            vp[page, :, row] = V[t]
        if q is not None:
            out[t], tq[t] = turn(f64(q)[t], at)
    return kp, vp, out, tk, tq


def same(got, want, tol):
    got = f64(got)
    assert (np.isnan(got) == np.isnan(want)).all()
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= tol[ok] + 0).all()


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 64, True), (96, 24, False), (96, 40, True), (128, 0, False)])
@pytest.mark.parametrize("order", ["phnd", "pnhd"])
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("lens", [[(1, 1)], [(1, 40 + i) for i in range(17)], [(100, 100), (0, 3), (1, 257), (33, 300)]],
                         ids=["first", "one", "chunk"])
def test_append(cuda_dev, D, rot, interleaved, order, page, lens):
    s = Step(lens, 6, 2, D, page, cuda_dev, seed=D, order=order, tail=5)
    r = pa.Rotary(rot, interleaved=interleaved, amplitude=0.5) if rot else None
    g = torch.Generator(device=cuda_dev).manual_seed(3)
    x = torch.randn(s.T, 10, D, generator=g, device=cuda_dev).bfloat16()  # one projection: q, k and v side by side
    q, k, v = x[:, :6], x[:, 6:8], x[:, 8:]
    kp, vp, out, tk, tq = append_want(s, k, v, q, r)
    got = torch.full((s.T, 6, D), 7.0, device=cuda_dev, dtype=torch.bfloat16)
    out[s.start[-1]:] = 7
    assert pa.paged_append(s.cache, q, k, v, *s.d, rotary=r, q_out=got) is got
    same(s.kp, kp, tk)
    same(s.vp, vp, np.zeros_like(vp))
    same(got, out, tq)


def test_append_positions_missing_places_in_place_and_without_queries(cuda_dev):
    s = Step([(4, 30), (3, 2), (5, 400), (2, 20)], 4, 2, 64, 16, cuda_dev, seed=21, width=20)
    s.table[0, 1] = -1         # the page of the first one's tokens 16 to 31
    s.table[3, :] = s.kp.shape[0]
    s.upload()                 # and the third one is longer than its row of the table
    r = pa.Rotary(32)
    g = torch.Generator(device=cuda_dev).manual_seed(4)
    q, k, v = (torch.randn(s.T, H, 64, generator=g, device=cuda_dev).bfloat16() for H in (4, 2, 2))
    pos = s.rng.integers(-1000, 100000, s.T).astype(np.int32)
    kp, vp, out, tk, tq = append_want(s, k, v, q, r, pos)
    before = s.kp.clone(), s.vp.clone()
    keep = q.clone()
    assert pa.paged_append(s.cache, q, k, v, *s.d, rotary=r, positions=torch.from_numpy(pos).to(cuda_dev), q_out=q) is q
    same(s.kp, kp, tk)
    same(s.vp, vp, np.zeros_like(vp))
    same(q, out, tq)
    after = s.kp.clone()
    s.kp.copy_(before[0])
    s.vp.copy_(before[1])
    assert pa.paged_append(s.cache, None, k, v, *s.d, rotary=r, positions=torch.from_numpy(pos).to(cuda_dev)) is None
    assert torch.equal(s.kp.nan_to_num(9), after.nan_to_num(9))
    assert torch.equal(pa.paged_append(s.cache, keep, k, v, *s.d, rotary=r, positions=torch.from_numpy(pos).to(cuda_dev)), q)


def test_many_sequences_append(cuda_dev):
    s = Step([((i * 5) % 3, (i * 5) % 3 + i % 30) for i in range(2500)], 2, 1, 64, 16, cuda_dev, seed=22, tail=1)
    g = torch.Generator(device=cuda_dev).manual_seed(5)
    k, v = (torch.randn(s.T, 1, 64, generator=g, device=cuda_dev).bfloat16() for _ in range(2))
    kp, vp, _, tk, _ = append_want(s, k, v, None, None)
    pa.paged_append(s.cache, None, k, v, *s.d)
    same(s.kp, kp, tk)
    same(s.vp, vp, np.zeros_like(vp))


# ------------------------------------------------------------- as they are used
def test_generation_is_the_packed_forward(cuda_dev):
    """Prompts in chunks, then token by token: the cache's keys are rotary_forward's to
    the bit, and the outputs those of the packed attention of the whole sequences."""
    Hq, Hkv, D, page = 8, 2, 128, 16
    lens, prompts = [150, 37, 260], [100, 1, 200]
    N = sum(lens)
    g = torch.Generator(device=cuda_dev).manual_seed(6)
    q, k, v = (torch.randn(1, N, H, D, generator=g, device=cuda_dev).bfloat16().transpose(1, 2) for H in (Hq, Hkv, Hkv))
    seg = torch.from_numpy(np.repeat(np.arange(3, dtype=np.int32), lens)[None]).to(cuda_dev)
    r = pa.Rotary(D, theta=5e5)
    qr, kr = pa.rotary_forward([q, k], r, pa.segment_positions(seg))
    want, wl = pa.forward(qr, kr, v, seg)
    first = np.concatenate([[0], np.cumsum(lens)])
    width = -(-max(lens) // page)
    pool = torch.full((3 * width, 2, Hkv, page, D), NAN, device=cuda_dev, dtype=torch.bfloat16)
    cache = pa.PagedCache(pool[:, 0], pool[:, 1])
    table = torch.randperm(3 * width, generator=g, device=cuda_dev).to(torch.int32).view(3, width)
    done = [0, 0, 0]
    while done != lens:
        new = [min(n - d, 70 if d < p else 1) for n, d, p in zip(lens, done, prompts)]
        rows = torch.cat([torch.arange(first[s] + done[s], first[s] + done[s] + new[s]) for s in range(3)]).to(cuda_dev)
        done = [d + n for d, n in zip(done, new)]
        start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=cuda_dev)
        kv = torch.tensor(done, dtype=torch.int32, device=cuda_dev)
        take = lambda x: x[0].transpose(0, 1)[rows]
        got = pa.paged_append(cache, take(q), take(k), take(v), table, start, kv, rotary=r)
        assert torch.equal(got, take(qr))
        out, lse = pa.paged_forward(got, cache, table, start, kv)
        # both are within half a step of the weights' and of the result's rounding of the same numbers
        assert (out.float() - take(want).float()).abs().max() <= 2e-2
        assert (lse - wl[0].T[rows]).abs().max() <= 1e-4
    for s in range(3):
        at = torch.arange(lens[s], device=cuda_dev)
        keys = cache.k[table[s].long()[at // page], :, at % page]
        assert torch.equal(keys, kr[0, :, first[s]:first[s + 1]].transpose(0, 1))


def test_captured_step_takes_new_lengths(cuda_dev):
    """Append and attention of a step in one graph, replayed as the sequences grow;
    two graphs share a workspace."""
    S, Hq, Hkv, D, page, width = 3, 4, 2, 64, 16, 30
    g = torch.Generator(device=cuda_dev).manual_seed(7)
    pool = torch.zeros(S * width, 2, Hkv, page, D, device=cuda_dev, dtype=torch.bfloat16)
    cache = pa.PagedCache(pool[:, 0], pool[:, 1])
    table = torch.randperm(S * width, generator=g, device=cuda_dev).to(torch.int32).view(S, width)
    start = torch.arange(S + 1, device=cuda_dev, dtype=torch.int32)
    kv = torch.tensor([3, 200, 470], device=cuda_dev, dtype=torch.int32)
    q, k, v = (torch.empty(S, H, D, device=cuda_dev, dtype=torch.bfloat16) for H in (Hq, Hkv, Hkv))
    r = pa.Rotary(D)
    ws = pa.paged_workspace(q, cache)
    pool.normal_(generator=g)
    graphs, outs = [], []
    for _ in range(2):
        qr, out = torch.empty_like(q), torch.empty_like(q)
        lse = torch.empty(S, Hq, device=cuda_dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pa.paged_append(cache, q, k, v, table, start, kv, rotary=r, q_out=qr)
            pa.paged_forward(qr, cache, table, start, kv, out=out, lse=lse, ws=ws)
        graphs.append(graph)
        outs.append((qr, out, lse))
    for i in range(6):
        for x in (q, k, v):
            x.normal_(generator=g)
        kv += torch.tensor([40, 1, 2], device=cuda_dev, dtype=torch.int32)
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        qr, out, lse = outs[i % 2]
        want, wl = pa.paged_forward(qr, cache, table, start, kv)
        assert torch.equal(out, want) and torch.equal(lse, wl) and torch.equal(qr, pa.paged_append(cache, q, k, v, table, start, kv, rotary=r))
        ref, rl, A, Z = paged.attention(f64(qr), f64(cache.k), f64(cache.v), table.cpu().numpy(), list(range(S + 1)), kv.cpu().numpy())
        assert (np.abs(f64(out) - ref) <= (2 * 2.0 ** -8 + 2.0 ** -11) * A + 2.0 ** -8 * np.abs(ref)).all()
    assert pa.pa_device_status(ws) == 0


def test_two_streams_at_once(cuda_dev):
    steps = [Step([(1, 5000), (64, 700)], 8, 2, 128, 64, cuda_dev, seed=30 + i) for i in range(2)]
    want = [s.forward() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    ws = [pa.paged_workspace(s.q, s.cache) for s in steps]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, (s, st) in enumerate(zip(steps, streams)):
            with torch.cuda.stream(st):
                got[i].append(pa.paged_forward(s.q, s.cache, *s.d, ws=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(a, b) for r in got[i] for a, b in zip(r, want[i]))


def test_offsets_past_32_bits(cuda_dev):
    """A cache of more than 2^31 elements a side, its last pages in use."""
    Hkv, page, D = 8, 256, 128
    pages = (1 << 31) // (Hkv * page * D) + 40
    kp, vp = (torch.full((pages, Hkv, page, D), NAN, device=cuda_dev, dtype=torch.bfloat16) for _ in range(2))
    ids = [pages - 1, 3, pages - 2, pages - 30]
    small = Step([(2, 900)], 8, Hkv, D, page, cuda_dev, seed=40, spare=0)
    for j, p in enumerate(ids):
        kp[p], vp[p] = small.kp[int(small.table[0, j])], small.vp[int(small.table[0, j])]
    want, wl = small.forward()
    big = pa.PagedCache(kp, vp)
    table = torch.tensor([ids], dtype=torch.int32, device=cuda_dev)
    out, lse = pa.paged_forward(small.q, big, table, *small.d[1:])
    assert torch.equal(out, want) and torch.equal(lse, wl)
    k, v = (torch.randn(2, Hkv, D, device=cuda_dev).bfloat16() for _ in range(2))
    pa.paged_append(big, None, k, v, table, *small.d[1:])
    assert torch.equal(kp[ids[3], :, 898 % page:900 % page].transpose(0, 1), k)
    assert torch.equal(vp[ids[3], :, 898 % page:900 % page].transpose(0, 1), v)


def test_no_rows(cuda_dev):
    s = Step([(0, 5)], 4, 2, 64, 16, cuda_dev)
    out, lse = pa.paged_forward(s.q, s.cache, *s.d)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    e = torch.empty(0, 2, 64, device=cuda_dev, dtype=torch.bfloat16)
    assert pa.paged_append(s.cache, s.q, e, e, *s.d).shape == (0, 4, 64)


def test_python_refusals(cuda_dev):
    s = Step([(2, 50)], 4, 2, 64, 16, cuda_dev)
    table, start, kv = s.d
    k = torch.zeros(2, 2, 64, device=cuda_dev, dtype=torch.bfloat16)
    for args, match in (((s.q.float(), s.cache, table, start, kv), "bfloat16"), ((s.q[..., :32], s.cache, table, start, kv), "must be"),
                        ((s.q, s.cache, table.long(), start, kv), "int32"), ((s.q, s.cache, table, start[:1], kv), "q_start"),
                        ((s.q, s.cache, table.cpu(), start, kv), "current CUDA device"), ((s.q[0], s.cache, table, start, kv), "must be"),
                        ((s.q, s.cache, table.repeat(1, 2)[:, ::2], start, kv), "contiguous")):
        with pytest.raises(ValueError, match=match):
            pa.paged_forward(*args, out=torch.empty_like(s.q), lse=torch.empty(2, 4, device=cuda_dev))
    with pytest.raises(ValueError, match="out must"):
        pa.paged_forward(s.q, s.cache, *s.d, lse=torch.empty(2, 3, device=cuda_dev))
    with pytest.raises(pa.PAError, match="PA_ERR_GQA"):
        pa.paged_forward(s.q[:, :3], s.cache, *s.d)
    with pytest.raises(pa.PAError, match="PA_ERR_WORKSPACE"):
        pa.paged_forward(s.q, s.cache, *s.d, ws=torch.empty(64, dtype=torch.uint8, device=cuda_dev))
    with pytest.raises(ValueError, match="k's shape and strides"):
        pa.paged_append(s.cache, None, k, torch.zeros(2, 4, 64, device=cuda_dev, dtype=torch.bfloat16)[:, ::2], *s.d)
    with pytest.raises(ValueError, match="come together"):
        pa.paged_append(s.cache, None, k, k, *s.d, q_out=s.q)
    with pytest.raises(ValueError, match="rows"):
        pa.paged_append(s.cache, s.q[:1], k, k, *s.d)
    with pytest.raises(ValueError, match="current CUDA device"):
        pa.paged_append(pa.PagedCache(s.kp.cpu(), s.vp.cpu()), None, k, k, *s.d)
