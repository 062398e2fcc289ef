"""Operators on rows of logits, written out in fp64: the token draw, the top
logits, and the distillation loss against a teacher's top logits with its
gradient. One row at a time, from the definitions.

The draw's raw and processed scores are the two "score definitions" of [AMD]
"Make Sure Both Scores Answer the Same Question" (top-k example: keeping two
of (0.5, 0.3, 0.2) renormalises them to (0.625, 0.375, 0)).
"""

from __future__ import annotations

import numpy as np


def _row_ok(z: np.ndarray) -> bool:
    return not np.isnan(z).any() and not np.isposinf(z).any() and np.isfinite(z).any()


def token_order(z: np.ndarray) -> np.ndarray:
    """Tokens by (logit descending, index ascending)."""
    return np.lexsort((np.arange(z.size), -z))


def sample_row(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, processed, kept) of one row; token -1 and NaN scores
    where there is no valid draw. Settings are fp32 values."""
    z = np.asarray(z, np.float64)
    tau, u, top_p, min_p = (float(np.float32(v)) for v in (temperature, u, top_p, min_p))
    tau_ok = tau == 0 or 2.0 ** -126 <= tau < np.inf
    if not _row_ok(z) or not tau_ok or np.isnan([u, top_p, min_p]).any():
        return -1, np.nan, np.nan, 0
    greedy = tau == 0
    order = token_order(z)
    s = z[order] / (1.0 if greedy else tau)
    w = np.exp(s - s[0])
    logprob = s - s[0] - np.log(w.sum())
    if greedy:
        return int(order[0]), float(logprob[0]), 0.0, 1
    kept = int(np.isfinite(z).sum())
    if top_k > 0:
        kept = min(kept, int(top_k))
    c = np.cumsum(w)
    if top_p < 1:
        want = top_p * c[kept - 1]
        kept = min(kept, 1 if want <= 0 else int(np.argmax(c >= want)) + 1)
    if min_p > 0:
        kept = max(1, min(kept, int((w >= min_p).sum())))
    u = min(max(u, 0.0), 1.0 - 2.0 ** -24)
    rank = int(np.argmax(c[:kept] > u * c[kept - 1]))
    return (int(order[rank]), float(logprob[rank]),
            float(s[rank] - s[0] - np.log(c[kept - 1])), kept)


def sample(z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """Rows of sample_row; settings are scalars or one per row."""
    n = len(u)
    b = [np.broadcast_to(v, (n,)) for v in (temperature, top_k, top_p, min_p)]
    out = [sample_row(z[i], u[i], b[0][i], b[1][i], b[2][i], b[3][i]) for i in range(n)]
    return (np.array([o[0] for o in out], np.int64), np.array([o[1] for o in out]),
            np.array([o[2] for o in out]), np.array([o[3] for o in out], np.int32))


def top_logprobs(z, k, temperature=1.0):
    """(ids, logits, logprobs, lse) of the k first tokens of every row."""
    z = np.asarray(z, np.float64)
    tau = float(np.float32(temperature))
    n = z.shape[0]
    ids = np.full((n, k), -1, np.int64)
    val = np.full((n, k), -np.inf)
    lp = np.full((n, k), -np.inf)
    lse = np.full(n, np.nan)
    for i in range(n):
        if not _row_ok(z[i]):
            val[i] = lp[i] = np.nan
            continue
        order = token_order(z[i])
        m = min(k, int(np.isfinite(z[i]).sum()))
        s = z[i] / tau
        log_sum = np.log(np.exp(s - s.max()).sum())
        lse[i] = s.max() + log_sum
        ids[i, :m] = order[:m]
        val[i, :m] = z[i][order[:m]]
        lp[i, :m] = s[order[:m]] - s.max() - log_sum  # (s - lse loses log_sum where s is large)
    return ids, val, lp, lse


def distill_row(z, ids, teacher, temperature=1.0, renormalize=True):
    """(loss, gradient [V]) of one row: the teacher's distribution spread over
    the vocabulary, its divergence from softmax(z / tau), and (Q p - q) / tau."""
    z = np.asarray(z, np.float64)
    tau = float(np.float32(temperature))
    V = z.size
    there = ids != -1
    ids, x = ids[there], np.asarray(teacher, np.float64)[there]
    nan = np.full(V, np.nan)
    if ((ids < 0) | (ids >= V)).any() or np.isnan(x).any() or np.isposinf(x).any():
        return np.nan, nan
    if x.size == 0 or np.isneginf(x).all():
        return 0.0, np.zeros(V)
    if renormalize:
        x = x / tau
        x = x - (x.max() + np.log(np.exp(x - x.max()).sum()))
    q = np.exp(x)
    if q.sum() == 0:
        return 0.0, np.zeros(V)
    if not _row_ok(z):
        return np.nan, nan
    s = z / tau
    logp = s - (s.max() + np.log(np.exp(s - s.max()).sum()))
    loss = sum(qk * (xk - logp[i]) for qk, xk, i in zip(q, x, ids) if qk > 0)
    target = np.zeros(V)
    np.add.at(target, ids, q)
    return float(loss), (q.sum() * np.exp(logp) - target) / tau


def distill(z, ids, teacher, temperature=1.0, renormalize=True, weight=None):
    """Rows of distill_row: (loss [T], weight * gradient [T, V]); a row of
    weight 0 has gradient 0."""
    T = len(z)
    rows = [distill_row(z[t], ids[t], teacher[t], temperature, renormalize) for t in range(T)]
    weight = np.ones(T) if weight is None else np.asarray(weight, np.float64)
    grad = [np.zeros_like(g) if weight[t] == 0 else weight[t] * g
            for t, (_, g) in enumerate(rows)]
    return np.array([r[0] for r in rows]), np.array(grad)
