"""Scores under the 8-bit head where 0 meets infinity: a token whose scale is 0 beside
rows of the head whose scale is infinite or no number."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import int8_head as oracle

from .gpu_helpers import DEV
from .logits_helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16_logits", [False, True])
@pytest.mark.parametrize("t", [5, 70, 200])
@pytest.mark.parametrize("v", [100, 256, 300, 8400, 16500])
@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
def test_zero_times_infinity(scale, v, t, bf16_logits):
    """A logit 0 x infinity is no number, so its row has no score, wherever in the
    vocabulary it lies: in a whole block of 128 rows or in the last, ragged one."""
    rng = np.random.default_rng(v + t)
    h = 64
    qx = rng.integers(-127, 128, (t, h)).astype(np.int8)
    qw = rng.integers(-127, 128, (v, h)).astype(np.int8)
    sx = (rng.random(t) * 1e-3 + 1e-4).astype(np.float32)
    sx[0], sx[1] = 0.0, -0.0
    # The place's sums are negative, 0 and positive by the token.
    for at in (0, v // 2, v - 1):
        sw = (rng.random(v) * 0.01).astype(np.float32)
        sw[at] = scale
        z = oracle.logits_f32(qx, sx, qw, sw)
        gone = (np.isnan(z) | np.isposinf(z)).any(axis=1)
        assert gone[:2].all()
        ids = rng.integers(0, v, t)
        ids[ids == at] = (at + 1) % v
        x, w = torch.from_numpy(qx).to(DEV), torch.from_numpy(qw).to(DEV)
        args = (x, dev(sx, torch.float32), w, dev(sw, torch.float32), dev(ids, torch.int64))
        lse = torch.empty(t, device=DEV)
        got = lp.score_int8(*args, bf16_logits=bf16_logits, lse=lse)
        assert np.array_equal(np.isnan(got.cpu().numpy()), gone)
        assert np.array_equal(np.isnan(lse.cpu().numpy()), gone)


@pytest.mark.parametrize("v", [100, 300, 8400])
def test_tokens_without_a_scale_score_all_alike(v):
    rng = np.random.default_rng(v)
    x = torch.randint(-127, 128, (70, 64), device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (v, 64), device=DEV, dtype=torch.int8)
    ws = dev(rng.random(v) * 1e30, torch.float32)
    got = lp.score_int8(x, torch.zeros(70, device=DEV), w, ws, dev(rng.integers(0, v, 70), torch.int64))
    # A sum of v equal terms: exact; its logarithm, and the last product.
    assert (got + np.log(v)).abs().max() <= 4 * 2.0 ** -24 * np.log(v)
