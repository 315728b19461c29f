"""What the rollouts of a policy add to its training on packed rows, as cases to
measure:

  rope_fwd   positions of packed rows from their segment ids, and queries and
             keys rotated by them
  rope_bwd   the gradients of the rotated queries and keys taken back
  append     new tokens' keys (rotated on the way) and values written into a
             paged cache, their queries rotated beside them
  paged      attention of the new tokens over the paged cache: one token a
             sequence, a few, whole chunks of a prompt, or a mixture

``run`` computes a case in plain torch operations (fp32, angles in fp64) when
``own`` is false and through segment_masked_causal_gb300 when it is true;
``exact`` gives the same outputs in fp64 from the definitions.

A case's lengths come from its number ``lens`` alone, so that ``work`` can
count them; the values and the order of the pages come from the seed.
"""
import math
import random

import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # the attention benchmark's packed 8k row, q and k as the projections leave them
        dict(name="rope_fwd_8k_packed", op="rope_fwd", B=1, Hq=32, Hkv=8, N=8192, D=128, rot=128, pairs="half",
             scaling="none", factor=1.0, dtype="bf16", layout="bnhd", lo=256, hi=2048, lens=1),
        # two short ragged rows in fp32, a quarter of each head, a context stretched four times
        dict(name="rope_fwd_f32_2x333", op="rope_fwd", B=2, Hq=16, Hkv=4, N=333, D=96, rot=24, pairs="interleaved",
             scaling="bands", factor=4.0, dtype="f32", layout="bhnd", lo=20, hi=200, lens=2),
        # the gradients of four packed rows, half of each head
        dict(name="rope_bwd_4x4096", op="rope_bwd", B=4, Hq=32, Hkv=8, N=4096, D=128, rot=64, pairs="half",
             scaling="linear", factor=2.0, dtype="bf16", layout="bhnd", lo=8, hi=1024, lens=3),
        # the running requests of a server, one token each
        dict(name="append_17", op="append", S=17, new="one", most=1, lo=1, hi=4000, Hq=32, Hkv=8, D=128, page=16,
             rot=128, pairs="half", tail=0, layout="phnd", lens=4),
        # prompts of ragged length, cut into one step of 8,000 tokens and padded
        dict(name="append_8000", op="append", S=7, new="chunk", most=8000, lo=0, hi=6000, Hq=32, Hkv=8, D=128, page=64,
             rot=128, pairs="half", tail=192, layout="pnhd", lens=5),
        # one request's next token, a short context: latency alone
        dict(name="paged_1", op="paged", S=1, new="one", most=1, lo=700, hi=700, Hq=32, Hkv=8, D=128, page=16, tail=0,
             layout="phnd", lens=6),
        # a batch of requests of very different age
        dict(name="paged_one_x64", op="paged", S=64, new="one", most=1, lo=30, hi=16000, Hq=32, Hkv=8, D=128, page=64,
             tail=0, layout="phnd", lens=7),
        # few long contexts, every query head with its own keys (the long rows of the attention benchmark)
        dict(name="paged_one_long", op="paged", S=3, new="one", most=1, lo=50000, hi=65536, Hq=8, Hkv=8, D=64, page=128,
             tail=0, layout="phnd", lens=8),
        # five guessed tokens a request checked at once, five query heads a key head
        dict(name="paged_few_x33", op="paged", S=33, new="few", most=5, lo=100, hi=6000, Hq=20, Hkv=4, D=96, page=16,
             tail=0, layout="pnhd", lens=9),
        # ragged prompts in one padded step of a smaller model
        dict(name="paged_chunk_1500", op="paged", S=4, new="chunk", most=1500, lo=0, hi=3500, Hq=16, Hkv=4, D=96, page=16,
             tail=36, layout="phnd", lens=10),
        # a chunk of a long prompt beside the other requests' tokens
        dict(name="paged_mixed_2048", op="paged", S=48, new="mixed", most=2048, lo=200, hi=9000, Hq=32, Hkv=8, D=128,
             page=32, tail=17, layout="pnhd", lens=11),
        # the second half of an 8k prompt
        dict(name="paged_chunk_4096", op="paged", S=1, new="chunk", most=4096, lo=8192, hi=8192, Hq=32, Hkv=8, D=128,
             page=64, tail=0, layout="phnd", lens=12),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    lens = rng.randrange(1 << 30)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq, D = Hkv * rng.choice([1, 2, 4, 4, 5, 7, 8]), rng.choice([64, 96, 128])
    Hq = min(Hq, 32) // Hkv * Hkv
    op = rng.choice(["rope_fwd", "rope_bwd", "append", "append", "paged", "paged", "paged", "paged"])
    pairs = rng.choice(["half", "interleaved"])
    if op in ("rope_fwd", "rope_bwd"):
        B = rng.randint(1, 4)
        lo = _log(rng, 1, 300)
        return dict(op=op, B=B, Hq=Hq, Hkv=Hkv, N=_log(rng, 1, 16384 // B), D=D, rot=rng.choice([16, 24, 32, 64, D, D]),
                    pairs=pairs, scaling=rng.choice(["none", "linear", "base", "bands"]),
                    factor=rng.choice([2.0, 4.0, 8.0]), dtype=rng.choice(["bf16", "bf16", "f32"]),
                    layout=rng.choice(["bnhd", "bhnd"]), lo=lo, hi=lo * rng.choice([1, 4, 16]), lens=lens)
    new = rng.choice(["one", "few", "chunk", "mixed"])
    S = _log(rng, 1, 64) if new in ("one", "few") else _log(rng, 1, 24)
    most = {"one": 1, "few": rng.randint(2, 9), "chunk": _log(rng, S, 4096), "mixed": _log(rng, S, 2048)}[new]
    hi = _log(rng, 20, 8192 if new in ("chunk", "mixed") else 300000 // S)
    case = dict(op=op, S=S, new=new, most=most, lo=rng.choice([0, 1, hi // 10, hi]), hi=hi, Hq=Hq, Hkv=Hkv, D=D,
                page=rng.choice([16, 32, 64, 128, 256]), tail=rng.choice([0, 0, rng.randint(1, 50)]),
                layout=rng.choice(["phnd", "pnhd"]), lens=lens)
    if op == "append":
        case.update(rot=rng.choice([16, 24, 32, D, D]), pairs=pairs)
    return case


def _lengths(case):
    """(new tokens, cached tokens with the new ones) of each sequence."""
    rng = random.Random(case["lens"])
    S, most, lo, hi = case["S"], case["most"], case["lo"], case["hi"]
    if case["new"] in ("one", "few"):
        new = [most] * S
    elif case["new"] == "mixed":
        new = [1] * S
        new[rng.randrange(S)] = max(1, most - S + 1)
    else:
        # `most` tokens cut at random places; a sequence may have none
        cuts = sorted(rng.randrange(most + 1) for _ in range(S - 1))
        new = [b - a for a, b in zip([0] + cuts, cuts + [most])]
    total = [max(n, _log(rng, max(1, lo), max(1, hi))) if n or lo else 0 for n in new]
    return list(zip(new, total))


def _segments(case):
    """Lengths of each row's segments, uniform in [lo, hi], until it is full."""
    rng, rows = random.Random(case["lens"]), []
    for _ in range(case["B"]):
        row, left = [], case["N"]
        while left:
            row.append(min(left, rng.randint(case["lo"], case["hi"])))
            left -= row[-1]
        rows.append(row)
    return rows


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("rope_fwd", "rope_bwd"):
        rows = case["B"] * case["N"]
        size = 2 if case["dtype"] == "bf16" else 4
        ids = 8 if case["op"] == "rope_fwd" else 4  # ids in and positions out, or positions in
        return {"bytes": 2 * rows * (Hq + Hkv) * D * size + ids * rows, "flops": 3 * rows * (Hq + Hkv) * case["rot"]}
    lens = _lengths(case)
    tokens = sum(n for n, _ in lens)
    tables = 4 * (2 * case["S"] + 1)
    if case["op"] == "append":
        return {"bytes": 4 * tokens * (Hq + 2 * Hkv) * D + tables, "flops": 3 * tokens * (Hq + Hkv) * case["rot"]}
    pairs = sum(n * t - n * (n - 1) // 2 for n, t in lens)
    keys = sum(t for n, t in lens if n)
    return {"bytes": 4 * keys * Hkv * D + 4 * tokens * Hq * D + 4 * tokens * Hq + tables
            + 4 * sum(-(-t // case["page"]) for n, t in lens if n), "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------ the inputs
THETA, ORIGINAL, LOW, HIGH = 10000.0, 2048, 1.0, 32.0


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 29)


def _frequencies(rot, scaling, factor):
    """Angle per position of each pair, and the factor on its cosine and sine."""
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=DEV)
    if scaling == "base":  # a larger base: the slowest pair stretched by the factor, the fastest not at all
        return (THETA * factor ** (rot / (rot - 2))) ** (-i / rot), 1.0
    f = THETA ** (-i / rot)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "bands":  # by how many turns a pair makes over the original context
        keep = ((ORIGINAL * f / (2 * math.pi) - LOW) / (HIGH - LOW)).clamp(0, 1)
        return f / factor * (1 - keep) + f * keep, 0.1 * math.log(factor) + 1
    return f, 1.0


def _rows(shape, layout, g, dtype):
    """(B, H, N, D) normals, contiguous or as a view of (B, N, H, D) memory."""
    B, H, N, D = shape
    if layout == "bnhd":
        return torch.randn(B, N, H, D, generator=g, device=DEV).to(dtype).transpose(1, 2)
    return torch.randn(B, H, N, D, generator=g, device=DEV).to(dtype)


def prepare(case, seed):
    s, g = dict(case), _gen(seed)
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] in ("rope_fwd", "rope_bwd"):
        s["freq"], s["amplitude"] = _frequencies(case["rot"], case["scaling"], case["factor"])
        s["frequencies"] = s["freq"].tolist()  # a model's program has them on the host
        dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        s["x"] = [_rows((case["B"], H, case["N"], D), case["layout"], g, dtype) for H in (Hq, Hkv)]
        # ids of each run as the packer numbers them, from a first one that the seed sets
        ids = [[i for i, n in enumerate(row) for _ in range(n)] for row in _segments(case)]
        s["seg"] = torch.tensor(ids, dtype=torch.int32, device=DEV) + int(seed) % 7
        if case["op"] == "rope_bwd":
            s["positions"] = torch.tensor([[i for n in row for i in range(n)] for row in _segments(case)],
                                          dtype=torch.int32, device=DEV)
        return s
    S, page = case["S"], case["page"]
    s["lengths"] = lens = _lengths(case)
    T = sum(n for n, _ in lens) + case["tail"]
    starts = [0]
    for n, _ in lens:
        starts.append(starts[-1] + n)
    s["q_start"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
    s["kv_len"] = torch.tensor([t for _, t in lens], dtype=torch.int32, device=DEV)
    # the pages of a pool in use by others too, in the order in which they were given out
    need = [-(-t // page) for _, t in lens]
    pages = sum(need) + 1 + sum(need) // 8
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    width = max(need) + 1
    table = torch.zeros(S, width, dtype=torch.int32)
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor(order[:n], dtype=torch.int32)
        del order[:n]
    s["table"] = table.to(DEV)

    def pool():
        shape = (pages, Hkv, page, D) if case["layout"] == "phnd" else (pages, page, Hkv, D)
        x = torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)
        return x if case["layout"] == "phnd" else x.transpose(1, 2)

    s["k_pages"], s["v_pages"] = pool(), pool()
    # one projection's rows: queries, keys and values side by side
    x = torch.randn(T, Hq + 2 * Hkv, D, generator=g, device=DEV, dtype=torch.bfloat16)
    if case["op"] == "append":
        s["q"], s["k"], s["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        s["freq"], s["amplitude"] = _frequencies(case["rot"], "none", 1.0)
        s["frequencies"] = s["freq"].tolist()
    else:
        s["q"] = x[:, :Hq].contiguous()
        s["lse"] = torch.zeros(T, Hq, device=DEV)
    s["out"] = torch.zeros(T, Hq, D, device=DEV, dtype=torch.bfloat16)  # rows behind the last sequence stay as they are
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    return {"rope_fwd": _run_rope, "rope_bwd": _run_rope, "append": _run_append, "paged": _run_paged}[s["op"]](s)


def _kept(s, name, make):
    """What a program makes once and keeps beside its tensors: handles and workspaces."""
    if name not in s:
        s[name] = make()
    return s[name]


def _rotary(s):
    import segment_masked_causal_gb300 as pa
    return _kept(s, "rotary", lambda: pa.Rotary(s["rot"], frequencies=s["frequencies"], amplitude=s["amplitude"],
                                                interleaved=s["pairs"] == "interleaved"))


def _rotate(x, pos, s, sign=1.0):
    """x (..., D) fp32 turned by pos (broadcast over x's heads) times the frequencies."""
    angle = pos.double()[..., None] * s["freq"]
    c, d = (angle.cos() * s["amplitude"]).float(), (angle.sin() * (sign * s["amplitude"])).float()
    rot = s["rot"]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if s["pairs"] == "interleaved" else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = [a * c - b * d, b * c + a * d]
    y = torch.stack(y, -1).flatten(-2) if s["pairs"] == "interleaved" else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _run_rope(s):
    fwd = s["op"] == "rope_fwd"
    if own:
        import segment_masked_causal_gb300 as pa
        if fwd:
            positions = pa.segment_positions(s["seg"])
            return {"positions": positions, "y": pa.rotary_forward(s["x"], _rotary(s), positions)}
        return {"dx": pa.rotary_backward(s["x"], _rotary(s), s["positions"])}
    if not fwd:
        return {"dx": [_rotate(x.float(), s["positions"][:, None], s, -1.0).to(x.dtype) for x in s["x"]]}
    seg, N = s["seg"], s["N"]
    n = torch.arange(N, device=seg.device)
    first = torch.ones_like(seg, dtype=torch.bool)
    first[:, 1:] = seg[:, 1:] != seg[:, :-1]
    start = torch.where(first, n, torch.zeros_like(n)).cummax(1).values
    positions = (n - start).int()
    return {"positions": positions, "y": [_rotate(x.float(), positions[:, None], s).to(x.dtype) for x in s["x"]]}


def _run_append(s):
    if own:
        import segment_masked_causal_gb300 as pa
        cache = _kept(s, "cache", lambda: pa.PagedCache(s["k_pages"], s["v_pages"]))
        pa.paged_append(cache, s["q"], s["k"], s["v"], s["table"], s["q_start"], s["kv_len"], _rotary(s), q_out=s["out"])
        return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    start, kv = s["q_start"].long(), s["kv_len"].long()
    T, page = s["q"].shape[0] - s["tail"], s["page"]
    t = torch.arange(T, device=start.device)
    seq = torch.searchsorted(start[1:], t, right=True)
    slot = kv[seq] - start[seq + 1] + t
    at = s["table"][seq, slot // page].long()
    s["out"][:T] = _rotate(s["q"][:T].float(), slot[:, None], s).bfloat16()
    s["k_pages"][at, :, slot % page] = _rotate(s["k"][:T].float(), slot[:, None], s).bfloat16()
    s["v_pages"][at, :, slot % page] = s["v"][:T]
    return {"q": s["out"], "k_pages": s["k_pages"], "v_pages": s["v_pages"]}


def _attend(q, k, v, total):
    """q (S, n, Hkv, G, D), k and v (S, L, Hkv, D), total (S,): the last of a
    sequence's n tokens sees its first total keys, the one before it one less."""
    n, L = q.shape[1], k.shape[1]
    S = torch.einsum("snhgd,slhd->shgnl", q, k) * (1 / math.sqrt(q.shape[-1]))
    last = total[:, None] - n + torch.arange(n, device=q.device)
    seen = torch.arange(L, device=q.device) <= last[..., None]
    S = S.masked_fill_(~seen[:, None, None], -math.inf)
    lse = S.amax(-1, keepdim=True)
    S = S.sub_(lse).exp_()
    total = S.sum(-1, keepdim=True)
    out = torch.einsum("shgnl,slhd->snhgd", S, v) / total.permute(0, 3, 1, 2, 4)
    return out.flatten(2, 3), (lse + total.log())[..., 0].permute(0, 3, 1, 2).flatten(2)


def _run_paged(s):
    if own:
        import segment_masked_causal_gb300 as pa
        cache = _kept(s, "cache", lambda: pa.PagedCache(s["k_pages"], s["v_pages"]))
        ws = _kept(s, "ws", lambda: pa.paged_workspace(s["q"], cache))
        pa.paged_forward(s["q"], cache, s["table"], s["q_start"], s["kv_len"], out=s["out"], lse=s["lse"], ws=ws)
        return {"out": s["out"], "lse": s["lse"]}
    Hkv, page, lens = s["Hkv"], s["page"], s["lengths"]
    q = s["q"].unflatten(1, (Hkv, -1))

    def gather(x, rows, width):  # (S, keys, Hkv, D) of some rows of the table
        return x[s["table"][rows, :width].long()].transpose(2, 3).flatten(1, 2).float()

    if s["new"] in ("one", "few"):  # all sequences at once, filled up to the longest
        n = s["most"]
        width = -(-max(t for _, t in lens) // page)
        out, lse = _attend(q[:n * len(lens)].float().unflatten(0, (-1, n)), gather(s["k_pages"], slice(None), width),
                           gather(s["v_pages"], slice(None), width), s["kv_len"])
        s["out"][:n * len(lens)] = out.flatten(0, 1).bfloat16()
        s["lse"][:n * len(lens)] = lse.flatten(0, 1)
        return {"out": s["out"], "lse": s["lse"]}
    at = 0
    for i, (n, t) in enumerate(lens):
        if n:
            rows, width = slice(i, i + 1), -(-t // page)
            out, lse = _attend(q[None, at:at + n].float(), gather(s["k_pages"], rows, width)[:, :t],
                               gather(s["v_pages"], rows, width)[:, :t], s["kv_len"][rows])
            s["out"][at:at + n] = out[0].bfloat16()
            s["lse"][at:at + n] = lse[0]
        at += n
    return {"out": s["out"], "lse": s["lse"]}


# ------------------------------------------------------------------ in 64 bits
#: Products that fp64 does in about ten seconds.
EXACT_FLOPS = 6e12


def exact(case, seed):
    if work(case)["flops"] > EXACT_FLOPS:
        return None
    return {"rope_fwd": _exact_rope, "rope_bwd": _exact_rope, "append": _exact_append, "paged": _exact_paged}[case["op"]](
        prepare(case, seed))


def _turn(x, pos, s, back=False):
    """Pairs of x (..., H, D) as complex numbers times amplitude * exp(i pos f); pos of x's shape without its last two."""
    half, D = s["rot"] // 2, x.shape[-1]
    pairs = list(range(0, 2 * half, 2)) if s["pairs"] == "interleaved" else list(range(half))
    mates = [p + 1 for p in pairs] if s["pairs"] == "interleaved" else [p + half for p in pairs]
    y = x.double().clone()
    z = torch.complex(y[..., pairs], y[..., mates])
    phase = pos.double()[..., None, None] * torch.tensor(s["frequencies"], dtype=torch.float64, device=x.device)
    z = z * torch.polar(torch.full_like(phase, s["amplitude"]), -phase if back else phase)
    y[..., pairs], y[..., mates] = z.real, z.imag
    return y


def _exact_rope(s):
    if s["op"] == "rope_bwd":
        return {"dx": [_turn(x.transpose(1, 2), s["positions"], s, back=True).transpose(1, 2) for x in s["x"]]}
    pos = torch.tensor([[i for n in row for i in range(n)] for row in _segments(s)], dtype=torch.int32, device=DEV)
    return {"positions": pos, "y": [_turn(x.transpose(1, 2), pos, s).transpose(1, 2) for x in s["x"]]}


def _exact_append(s):
    out, k, v = s["out"].double(), s["k_pages"].double(), s["v_pages"].double()
    at = 0
    for i, (n, t) in enumerate(s["lengths"]):
        if n:
            pos = torch.arange(t - n, t, device=DEV)
            where = (s["table"][i].long()[pos // s["page"]], slice(None), pos % s["page"])
            out[at:at + n] = _turn(s["q"][at:at + n], pos, s)
            k[where] = _turn(s["k"][at:at + n], pos, s)
            v[where] = s["v"][at:at + n].double()
        at += n
    return {"q": out, "k_pages": k, "v_pages": v}


def _exact_paged(s):
    out, lse = s["out"].double(), s["lse"].double()
    Hq, G, page, at = s["Hq"], s["Hq"] // s["Hkv"], s["page"], 0
    for i, (n, t) in enumerate(s["lengths"]):
        ids = s["table"][i, :-(-t // page)].long()
        for h in range(s["Hkv"] if n else 0):
            k, v = (x[ids, h].reshape(-1, s["D"])[:t].double() for x in (s["k_pages"], s["v_pages"]))
            future = torch.ones(n, t, dtype=torch.bool, device=DEV).triu(t - n + 1)
            for hq in range(h * G, (h + 1) * G):
                z = (s["q"][at:at + n, hq].double() @ k.T / math.sqrt(s["D"])).masked_fill(future, -math.inf)
                lse[at:at + n, hq] = torch.logsumexp(z, 1)
                out[at:at + n, hq] = torch.softmax(z, 1) @ v
        at += n
    return {"out": out, "lse": lse}
