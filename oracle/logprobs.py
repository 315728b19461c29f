"""fp64 restatement of the token log probabilities (test infrastructure).

TEST INFRASTRUCTURE ONLY: only the tests may import this module; the library
never calls it and shares no code with it.

    z_iv   = <H_i, W_v> / T
    lse_i  = log sum_v exp(z_iv)           p_iv = exp(z_iv - lse_i)
    logp_i = z_{i, t_i} - lse_i            (0 where t_i lies outside [0, V))
    ent_i  = -sum_v p_iv log p_iv
    alternatives: the K largest z_iv, the lower v first among equals
    L      = sum_i g_i logp_i + e_i ent_i:
    dz_iv  = (g_i ([v == t_i] - p_iv) - e_i p_iv (log p_iv + ent_i)) / T
    dH     = dz W,   dW = dz^T H           (an unscored token's g_i counts as 0)

Pins: tests/test_logprobs_host.py (torch float64 log_softmax with autograd,
central finite differences, uniform and single-entry vocabularies, ties).
"""
from __future__ import annotations

import numpy as np


def _log_softmax(H, W, T):
    z = (np.asarray(H, np.float64) @ np.asarray(W, np.float64).T) / T
    m = z.max(axis=1, keepdims=True)
    lse = m + np.log(np.exp(z - m).sum(axis=1, keepdims=True))
    return z - lse, lse[:, 0]


def forward(H, W, targets, T=1.0, top=0):
    """(logp, lse, entropy, ids, alt): ids and alt (N, top)."""
    lp, lse = _log_softmax(H, W, T)
    N, V = lp.shape
    t = np.asarray(targets, np.int64)
    scored = (t >= 0) & (t < V)
    logp = np.where(scored, lp[np.arange(N), np.where(scored, t, 0)], 0.0)
    p = np.exp(lp)
    entropy = -np.where(p > 0, p * lp, 0.0).sum(axis=1)
    raw = np.asarray(H, np.float64) @ np.asarray(W, np.float64).T
    order = np.argsort(-raw, axis=1, kind="stable")[:, :top]
    return logp, lse, entropy, order, np.take_along_axis(lp, order, axis=1)


def backward(H, W, targets, g, e, T=1.0):
    """(dH, dW) for the upstream g = dL/dlogp and e = dL/dentropy (or None)."""
    lp, _ = _log_softmax(H, W, T)
    N, V = lp.shape
    t = np.asarray(targets, np.int64)
    scored = (t >= 0) & (t < V)
    p = np.exp(lp)
    gs = np.where(scored, np.asarray(g, np.float64), 0.0)
    dz = -gs[:, None] * p
    dz[np.arange(N)[scored], t[scored]] += gs[scored]
    if e is not None:
        ent = -np.where(p > 0, p * lp, 0.0).sum(axis=1)
        dz -= np.asarray(e, np.float64)[:, None] * p * (np.where(p > 0, lp, 0.0) + ent[:, None])
    dz /= T
    return dz @ np.asarray(W, np.float64), dz.T @ np.asarray(H, np.float64)
