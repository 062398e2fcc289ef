"""Calls of the operators on rows of logits that their documentation allows
beside the plain ones: counters and scratch memory of the caller's."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .gpu_helpers import DEV
from .logits_helpers import rows

pytestmark = pytest.mark.gpu


def test_checked_calls_with_a_counter_that_is_not_zero():
    t, _ = rows(4, 6, 700)
    wrong = t.clone()
    wrong[2, 5] = wrong[4, 6] = float("nan")
    u = torch.full((6,), 0.5, device=DEV)
    ids = torch.zeros(6, 3, dtype=torch.int64, device=DEV)
    outside = ids.clone()
    outside[1, 2] = outside[5, 0] = 700
    x, w = torch.zeros(6, 3, device=DEV), torch.ones(6, device=DEV)
    calls = [(lambda bad, z: lp.sample(z, u, top_k=5, bad_rows=bad, check=True), t, wrong),
             (lambda bad, z: lp.sample(z, u, top_p=0.9, bad_rows=bad, check=True), t, wrong),
             (lambda bad, z: lp.top_logprobs(z, 5, bad_rows=bad, check=True), t, wrong),
             (lambda bad, i: lp.distill_forward(t, i, x, bad_rows=bad, check=True), ids, outside),
             (lambda bad, i: lp.distill_step(t, i, x, w, bad_rows=bad, check=True), ids, outside)]
    for call, clean, broken in calls:
        bad = torch.full((1,), 3, dtype=torch.int32, device=DEV)
        call(bad, clean)
        assert bad.item() == 3
        with pytest.raises(ValueError, match="^2 row"):
            call(bad, broken)
        assert bad.item() == 5
    bad = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    lp.sample(wrong, u, top_k=5, bad_rows=bad)
    lp.top_logprobs(wrong, 5, bad_rows=bad)
    assert bad.item() == 7
