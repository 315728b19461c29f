"""A paged cache and the attention over it in fp64, token by token from the
definitions."""
import math

import numpy as np


def places(q_start, kv_len, table, pages, page):
    """(row, sequence, position, page or -1, row in the page) of each of a step's rows that has a sequence."""
    out = []
    for s in range(len(kv_len)):
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            pos = int(kv_len[s]) - n + i
            at = -1
            if pos >= 0 and pos // page < table.shape[1] and 0 <= table[s, pos // page] < pages:
                at = int(table[s, pos // page])
            out.append((int(q_start[s]) + i, s, pos, at, pos % page))
    return out


def attention(q, k_pages, v_pages, table, q_start, kv_len, scale=None):
    """q (T, Hq, D); pages (pages, Hkv, page, D). Returns out and lse (rows of no
    sequence NaN), A = sum_j w_j |v_j| per element and Z = the largest sum_c |q_c k_c| * scale
    per (row, head): what rounding errors scale with."""
    T, Hq, D = q.shape
    pages, Hkv, page, _ = k_pages.shape
    scale = scale or 1 / math.sqrt(D)
    out, A = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, Z = np.full((T, Hq), np.nan), np.zeros((T, Hq))
    for s in range(len(kv_len)):
        ids = [(j, int(table[s, j // page])) for j in range(min(int(kv_len[s]), table.shape[1] * page))]
        ids = [(j, p) for j, p in ids if 0 <= p < pages]
        keys = np.array([j for j, _ in ids], int)
        K = np.array([k_pages[p, :, j % page] for j, p in ids]).reshape(len(ids), Hkv, D)
        V = np.array([v_pages[p, :, j % page] for j, p in ids]).reshape(len(ids), Hkv, D)
        n = q_start[s + 1] - q_start[s]
        for i in range(n):
            t, see = q_start[s] + i, keys <= kv_len[s] - n + i
            if not see.any():
                out[t], lse[t] = 0, -np.inf
                continue
            for h in range(Hq):
                kk, vv = K[see, h // (Hq // Hkv)], V[see, h // (Hq // Hkv)]
                z = kk @ q[t, h] * scale
                top = z.max()
                w = np.exp(z - top)
                lse[t, h] = top + math.log(w.sum())
                w /= w.sum()
                out[t, h], A[t, h] = w @ vv, w @ np.abs(vv)
                Z[t, h] = (np.abs(kk) @ np.abs(q[t, h])).max() * scale
    return out, lse, A, Z
