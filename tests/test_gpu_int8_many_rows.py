"""Scores under the 8-bit head for more rows, times vocabulary, than a dispatch of a
workgroup for each tile would hold."""

import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bf16_logits", [False, True])
def test_a_million_rows(bf16_logits):
    """Rows that repeat: each has the bits that it has in a small batch."""
    g = torch.Generator(device=DEV).manual_seed(1)
    n, rows, v, h = 1009, 1000003, 151936, 64
    x = torch.randint(-127, 128, (n, h), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (v, h), generator=g, device=DEV, dtype=torch.int8)
    xs = torch.rand(n, generator=g, device=DEV) * 1e-3
    ws = torch.rand(v, generator=g, device=DEV) * 0.1
    ids = torch.randint(0, v, (n,), generator=g, device=DEV)
    lse = torch.empty(n, device=DEV)
    few = lp.score_int8(x, xs, w, ws, ids, bf16_logits=bf16_logits, lse=lse, check=True)
    assert torch.isfinite(few).all()
    at = torch.arange(rows, device=DEV) % n
    many_lse = torch.empty(rows, device=DEV)
    many = lp.score_int8(x[at], xs[at], w, ws, ids[at], bf16_logits=bf16_logits, lse=many_lse,
                         check=True)
    assert torch.equal(many, few[at]) and torch.equal(many_lse, lse[at])
