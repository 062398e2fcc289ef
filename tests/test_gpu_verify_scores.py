"""Scores of drafted tokens' verification (lp_verify) and of token draws (lp_sample) as
logarithms of probabilities: never above 0, and of rows that are summed whole to fp32's
one rounding."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import verify as oracle

from .logits_helpers import TYPES, dev, place, rows

pytestmark = pytest.mark.gpu

E = 2.0 ** -24

SETTINGS = [dict(), dict(temperature=0.7), dict(min_p=0.05), dict(top_p=0.9),
            dict(top_p=0.3, min_p=0.2), dict(top_k=5), dict(top_k=300),
            dict(top_k=300, top_p=0.8), dict(temperature=0.0)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("how", SETTINGS, ids=str)
def test_certain_tokens_of_drafts(how, dtype):
    """One token that holds all the weight, at logits whose fractions run over what
    the exponential is formed from; and rows of that token alone."""
    b, v = 257, 900
    z = np.full((2 * b, v), -np.inf)
    z[:, 1:40] = -3000.0
    z[:, 7] = np.arange(2 * b) * (8.0 / b) - 5.0
    ids, u = np.full((b, 1), 7), dev(np.full((b, 2), 0.5), torch.float32)
    for logits, drafted in ((place(z, dtype)[0], ids), (place(z[:, 7:8], dtype)[0], ids * 0)):
        tokens, accepted, raw, proc = lp.verify(logits, dev(drafted, torch.int64), u, **how)
        assert (tokens == int(drafted[0, 0])).all() and (accepted == 1).all()
        assert (raw <= 0).all() and (proc <= 0).all()


WHOLE = [dict(), dict(temperature=0.7), dict(min_p=0.05), dict(temperature=1.5, min_p=0.3),
         dict(temperature=0.01)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("v", [1, 2, 300, 9001])
@pytest.mark.parametrize("how", WHOLE, ids=str)
def test_rows_summed_whole(how, v, dtype):
    """Every weight within 1.1e-12 relative, so their sum's logarithm too, of the
    kernel's; what fp64 rounds besides is below 2^-40 at logits of these sizes; then
    fp32's half a step. Rows with a near-certain token among them."""
    b, d = 6, 2
    z, exact = rows(v, b * (d + 1), v, dtype)
    z[::2, v // 2] += 30
    exact = z.double().cpu().numpy()
    y, exact_y = place(exact.reshape(b, d + 1, v)[:, :d].reshape(b * d, v) + 0.1, dtype)
    ids = exact_y.argmax(axis=1).reshape(b, d)
    u = np.random.default_rng(v).random((b, d + 1)).astype(np.float32)
    got = lp.verify(z, dev(ids, torch.int64), dev(u, torch.float32), y, **how)
    want = oracle.verify(exact, ids, u, exact_y, **how)
    tokens, accepted, *scores = (t.cpu().numpy() for t in got)
    assert np.array_equal(tokens, want[0]) and np.array_equal(accepted, want[1])
    for score, ref in zip(scores, want[2:]):
        assert (np.abs(score - ref) <= E * np.abs(ref) + 1.1e-12 + 2.0 ** -40).all()


@pytest.mark.parametrize("gap", [20.0, 23.0, 26.0])
@pytest.mark.parametrize("how", [dict(), dict(top_p=0.5), dict(top_k=500, top_p=0.5),
                                 dict(top_p=0.5, temperature=0.8)], ids=str)
def test_certain_tokens_of_draws(how, gap):
    """A token so far above the others that a nucleus keeps it alone, in rows of buckets
    whose base is another token's logit."""
    rng = np.random.default_rng(int(gap))
    n, v = 200, 20011
    z = rng.normal(size=(n, v)) * 0.3
    z[np.arange(n), rng.integers(0, v, n)] = gap + 3 * rng.random(n)
    logits, _ = place(z)
    _, raw, proc, kept = lp.sample(logits, dev(rng.random(n) * 0.5, torch.float32), **how)
    assert (raw <= 0).all() and (proc <= 0).all()
    if "top_p" in how:
        assert (kept == 1).all() and (proc >= -1e-12).all()
