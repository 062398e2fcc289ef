"""Scores under the bf16 head of tokens that hold nearly all the weight, at logits of
hundreds and thousands: never above 0, by every entry point."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .gpu_helpers import DEV

pytestmark = pytest.mark.gpu


def peaked(seed, t, v, h, size):
    """Rows whose target's row of W is their own, scaled to logits around `size`."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randint(-127, 128, (t, h), generator=g, device=DEV).float()
    w = torch.randint(-127, 128, (v, h), generator=g, device=DEV).float()
    ids = torch.randperm(v, generator=g, device=DEV)[:t].contiguous()
    w[ids] = x
    scale = (0.5 + torch.rand(t, 1, generator=g, device=DEV)) * size / (5400 * h)
    return (x * scale).bfloat16(), w.bfloat16(), ids


@pytest.mark.parametrize("v", [500, 5000, 20011])
@pytest.mark.parametrize("t", [60, 400])
@pytest.mark.parametrize("temperature", [1.0, 0.7])
def test_no_score_lies_above_0(temperature, t, v):
    for seed, size in enumerate((30, 100, 200, 300, 1000, 1e5)):
        x, w, ids = peaked(seed, t, v, 64, size)
        got = lp.score(x, w, ids, temperature)
        assert torch.isfinite(got).all() and (got <= 0).all()
        # Every form has the same bits.
        stats, _, _ = lp.score_stats(x, w, ids, temperature)
        assert torch.equal(stats, got)
        parts = lp.shard_partials(t, False, DEV)
        for r in range(2):
            sh = lp.vocab_shard(v, 2, r)
            lp.score_shard(x, w[sh["row_begin"]:sh["row_end"]].clone(), ids, v, 2, r, parts,
                           temperature)
        assert torch.equal(lp.merge_shards(parts, ids, v), got)


def test_no_number_stays_none():
    x, w, ids = peaked(1, 60, 500, 64, 100)
    ids[3] = 500
    x[5] = float("nan")
    got = lp.score(x, w, ids)
    assert torch.isnan(got).nonzero().flatten().tolist() == [3, 5]
