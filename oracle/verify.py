"""Verification of drafted tokens, written out in fp64: one sequence at a time,
one position after the other, from the definition.

The distributions are lp_sample's (logit_rows.sample_row); scores answer the two
questions of [AMD] "Make Sure Both Scores Answer the Same Question".
"""

from __future__ import annotations

import numpy as np

from .logit_rows import _row_ok, token_order


def distribution(z, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(p [V], raw log-softmax [V]) of a row under fp32 settings: what lp_sample
    draws from. None where there is no valid draw."""
    z = np.asarray(z, np.float64)
    tau, top_p, min_p = (float(np.float32(v)) for v in (temperature, top_p, min_p))
    tau_ok = tau == 0 or 2.0 ** -126 <= tau < np.inf
    if not _row_ok(z) or not tau_ok or np.isnan([top_p, min_p]).any():
        return None
    order = token_order(z)
    s = (z - z[order[0]]) / (1.0 if tau == 0 else tau)
    w = np.exp(s[order])
    raw = s - np.log(w.sum())
    kept = int(np.isfinite(z).sum())
    if tau == 0:
        kept = 1
    else:
        if top_k > 0:
            kept = min(kept, int(top_k))
        c = np.cumsum(w)
        if top_p < 1:
            want = top_p * c[kept - 1]
            kept = min(kept, 1 if want <= 0 else int(np.argmax(c >= want)) + 1)
        if min_p > 0:
            kept = max(1, min(kept, int((w >= min_p).sum())))
    p = np.zeros(z.size)
    p[order[:kept]] = w[:kept] / w[:kept].sum()
    return p, raw


def verify_sequence(z, ids, u, y=None, **settings):
    """(tokens, accepted, logprob, processed) of one sequence: z [n + 1, V] the
    target's rows, ids [n], u [n + 1], y [n, V] the draft's rows or None."""
    n = len(ids)
    dists = [distribution(row, **settings) for row in z]
    drafts = [distribution(row, **settings) for row in y] if y is not None else []
    V = z.shape[1]
    if any(d is None for d in dists + drafts) or np.isnan(u).any() or \
            any(not 0 <= i < V for i in ids):
        return None
    u = np.clip(np.asarray(u, np.float64), 0.0, 1.0 - 2.0 ** -24)
    tokens, raws, procs = [], [], []
    for j in range(n + 1):
        p, raw = dists[j]
        weights = p
        if j < n:
            q = drafts[j][0] if y is not None else np.eye(1, V, ids[j])[0]
            if u[j] * q[ids[j]] < p[ids[j]]:
                tokens.append(int(ids[j]))
                raws.append(raw[ids[j]])
                procs.append(np.log(p[ids[j]]))
                continue
            weights = np.maximum(p - q, 0.0)
            if not weights.sum() > 0:
                weights = p
        c = np.cumsum(weights)
        t = int(np.argmax(c > u[n] * c[-1]))
        tokens.append(t)
        raws.append(raw[t])
        procs.append(np.log(p[t]))
        break
    return tokens, len(tokens) - 1, raws, procs


def verify(z, ids, u, y=None, counts=None, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Arrays as lp_verify lays them out: z [B (D + 1), V], ids [B, D], u
    [B, D + 1], y [B D, V] or None; settings are numbers or one per sequence."""
    B, D = ids.shape
    counts = np.full(B, D) if counts is None else counts
    how = [np.broadcast_to(v, (B,)) for v in (temperature, top_k, top_p, min_p)]
    tokens = np.full((B, D + 1), -1, np.int64)
    accepted = np.full(B, -1, np.int32)
    raw, proc = np.zeros((B, D + 1)), np.zeros((B, D + 1))
    for b in range(B):
        n = int(counts[b])
        got = None
        if 0 <= n <= D:
            rows = z[b * (D + 1):b * (D + 1) + n + 1]
            got = verify_sequence(rows, ids[b, :n], np.append(u[b, :n], u[b, D]),
                                  None if y is None else y[b * D:b * D + n],
                                  **dict(zip(("temperature", "top_k", "top_p", "min_p"),
                                             (h[b] for h in how))))
        if got is None:
            raw[b] = proc[b] = np.nan
            continue
        m = len(got[0])
        tokens[b, :m], accepted[b], raw[b, :m], proc[b, :m] = got
    return tokens, accepted, raw, proc
