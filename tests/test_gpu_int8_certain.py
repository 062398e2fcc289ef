"""Scores under the 8-bit head of tokens that hold nearly all the weight, at logits of
hundreds and thousands: never above 0, and as near as the sum's own rounding."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import int8_head as oracle

from .gpu_helpers import DEV

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def peaked(seed, t, v, h=64):
    """Codes where token i's target is a row of its own codes, its largest product."""
    rng = np.random.default_rng(seed)
    x = rng.integers(-127, 128, (t, h)).astype(np.int8)
    w = rng.integers(-127, 128, (v, h)).astype(np.int8)
    ids = rng.permutation(v)[:t]
    w[ids] = x
    return x, w, ids


def on(*arrays):
    return [torch.from_numpy(np.ascontiguousarray(a)).to(DEV) for a in arrays]


@pytest.mark.parametrize("bf16_logits", [False, True])
@pytest.mark.parametrize("v", [100, 300, 5000, 20011])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_no_score_lies_above_0(temperature, v, bf16_logits):
    t = 90
    x, w, ids = peaked(v, t, v)
    for size in (10, 100, 1000, 1e5):
        rng = np.random.default_rng(int(size))
        xs = (size * (0.5 + rng.random(t)) / 3.5e5).astype(np.float32)
        ws = np.full(v, np.float32(0.5 + rng.random()))
        args = on(x, xs, w, ws, ids.astype(np.int64))
        got = lp.score_int8(*args, temperature, bf16_logits=bf16_logits)
        assert torch.isfinite(got).all() and (got <= 0).all()


@pytest.mark.parametrize("v", [100, 300, 5000, 20011])
@pytest.mark.parametrize("power", [-14, -11, -9, -6])
def test_scores_beside_large_logits(power, v):
    """Scales are powers of two and the sums below 2^24, so the logits are exact, and what
    a score may be off by does not grow with them. With g the distance of a token's
    logit from the largest, p its probability and e = 2^-24: the factor log2(e) is
    rounded (e of every distance), a term's exponent and exponential are (e g and
    2 e of the term), a block adds 31 + 2 times and blocks are joined as in
    score_bound (6 e a step); then the score's rounding."""
    t = 90
    x, w, ids = peaked(v, t, v)
    xs, ws = np.full(t, np.float32(2.0 ** power)), np.ones(v, np.float32)
    lse = torch.empty(t, device=DEV)
    got = lp.score_int8(*on(x, xs, w, ws, ids.astype(np.int64)), lse=lse, check=True)
    z = oracle.logits(x, xs, w, ws)
    want, want_lse = oracle.log_softmax_at(z, ids)
    g = z.max(axis=1, keepdims=True) - z
    p = np.exp(z - want_lse[:, None])
    steps = -(-(-(-v // 128)) // 16) + 16
    bound = E * ((p * (3 + 2 * g)).sum(axis=1) + 33 + 6 * steps + 2 * np.abs(want))
    assert (got <= 0).all()
    assert (np.abs(got.cpu().numpy() - want) <= bound).all()
    # The log-sum has the factor's rounding at its full size, and its own.
    size = np.abs(z).max(axis=1)
    assert (np.abs(lse.cpu().numpy() - want_lse) <= bound + 2 * E * (size + 10)).all()
