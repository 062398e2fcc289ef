"""The LM head in 8-bit integers, written out in fp64: rows in 8 bits, rows of
logits and scores, from the definitions.

Integer sums are formed in int64, so they are exact; what the definition rounds
to fp32 (the scale, and each step from a sum to a logit) is rounded by numpy's
float32, which rounds to nearest even.
"""

from __future__ import annotations

import numpy as np


def quantize(x):
    """(codes int8 [R, H], scale fp32 [R]) of rows of finite or other values:
    a row with a NaN or an infinity has scale NaN and codes 0."""
    x = np.asarray(x, np.float32)
    codes = np.zeros(x.shape, np.int8)
    scale = np.full(x.shape[0], np.nan, np.float32)
    for r, row in enumerate(x):
        if not np.isfinite(row).all():
            continue
        scale[r] = np.abs(row).max() * (np.float32(1) / np.float32(127))
        if scale[r] > 0:
            ratio = row.astype(np.float64) / np.float64(scale[r])
            codes[r] = np.clip(np.rint(ratio), -127, 127).astype(np.int8)
    return codes, scale


def sums(x, w):
    """Exact sums of products [T, V]."""
    return np.asarray(x, np.int64) @ np.asarray(w, np.int64).T


def logits_f32(x, x_scale, w, w_scale):
    """Logits with the definition's roundings: the sum, and each product, to
    fp32."""
    with np.errstate(over="ignore", invalid="ignore"):
        z = sums(x, w).astype(np.float32) * np.asarray(x_scale, np.float32)[:, None]
        return z * np.asarray(w_scale, np.float32)[None, :]


def logits(x, x_scale, w, w_scale):
    """Logits without any rounding but fp64's."""
    return (sums(x, w).astype(np.float64) * np.asarray(x_scale, np.float64)[:, None]
            * np.asarray(w_scale, np.float64)[None, :])


def log_softmax_at(z, ids, temperature=1.0):
    """(logprob, lse) of the targets under rows of logits; a target outside the
    vocabulary gives NaN."""
    s = np.asarray(z, np.float64) / float(np.float32(temperature))
    top = s.max(axis=1)
    lse = top + np.log(np.exp(s - top[:, None]).sum(axis=1))
    ids = np.asarray(ids)
    ok = (ids >= 0) & (ids < s.shape[1])
    at = s[np.arange(len(ids)), np.where(ok, ids, 0)]
    return np.where(ok, at - lse, np.nan), lse
