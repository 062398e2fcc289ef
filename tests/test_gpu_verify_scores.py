"""Scores of drafted tokens' verification (lp_verify) and of token draws (lp_sample) as
logarithms of probabilities: never above 0."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .logits_helpers import TYPES, dev, place

pytestmark = pytest.mark.gpu

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
    for rows, drafted in ((place(z, dtype)[0], ids), (place(z[:, 7:8], dtype)[0], ids * 0)):
        tokens, accepted, raw, proc = lp.verify(rows, dev(drafted, torch.int64), u, **how)
        assert (tokens == int(drafted[0, 0])).all() and (accepted == 1).all()
        assert (raw <= 0).all() and (proc <= 0).all()
