"""Short lists of the token draw and the top logits that hold what they are
meant for: a list that overflows costs its row several more passes by one
workgroup. The slices' counts stand at the start of the scratch memory
(0xFFFFFFFF: overflowed)."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .gpu_helpers import DEV
from .logits_helpers import rows

pytestmark = pytest.mark.gpu
CODES = {"fp32": 0, "bf16": 1, "fp16": 2}


def overflows(call, name, n, v, dtype):
    """Slices (rows, where they are not cut) whose list overflowed in the call."""
    ws = torch.zeros(getattr(lp.lib(), name)(n, v, CODES[dtype]), dtype=torch.uint8, device=DEV)
    call(ws)
    chunks = -(-v // (512 * 4 * (4 if dtype == "fp32" else 8)))
    slices = max(1, min(chunks, 512 // n))
    return int((ws[:4 * n * slices].view(torch.int32) == -1).sum())


def count(t, n, v, dtype, k, draw):
    if draw:
        u = torch.full((n,), 0.5, device=DEV)
        return overflows(lambda ws: lp.sample(t, u, top_k=k, workspace=ws),
                         "lp_sample_workspace_bytes", n, v, dtype)
    return overflows(lambda ws: lp.top_logprobs(t, k, workspace=ws),
                     "lp_top_logprobs_workspace_bytes", n, v, dtype)


def test_a_list_that_does_overflow_is_seen():
    z = torch.zeros(2, 9001, device=DEV)
    assert count(z, 2, 9001, "fp32", 5, True) > 0 and count(z, 2, 9001, "fp32", 5, False) > 0


@pytest.mark.parametrize("dtype,n,v", [("bf16", 2, 2049), ("bf16", 3, 3000), ("fp16", 300, 3000),
                                       ("bf16", 300, 3583), ("fp32", 5, 2300), ("bf16", 1, 200064),
                                       ("bf16", 39, 200064), ("fp16", 2, 16384 * 2 + 2500)])
def test_a_chunk_that_the_row_ends_in(dtype, n, v):
    """Waves without a token of their own do not take the list's first bound away."""
    t, _ = rows(v + n, n, v, dtype)
    for k in (1, 20, 157):
        assert count(t, n, v, dtype, k, True) == 0, k
        assert count(t, n, v, dtype, k, False) == 0, k
    greedy = overflows(lambda ws: lp.sample(t, torch.zeros(n, device=DEV), 0.0, workspace=ws),
                       "lp_sample_workspace_bytes", n, v, dtype)
    assert greedy == 0


@pytest.mark.parametrize("dtype,n,v", [("fp16", 3, 9000), ("bf16", 2, 12001), ("fp32", 300, 6001)])
def test_many_wanted_of_a_chunk_that_the_row_ends_in(dtype, n, v):
    t, _ = rows(v + n, n, v, dtype)
    for k in (257, 300, 400):
        assert count(t, n, v, dtype, k, True) == 0, k
        assert count(t, n, v, dtype, k, False) == 0, k


@pytest.mark.parametrize("n", [2, 300])
def test_more_top_logits_than_a_list_are_not_collected(n):
    """Longer lists than collect_kernel makes go by buckets at once: no slice is
    collected and given up."""
    t, _ = rows(n, n, 20011, "bf16")
    for k in (421, 513, 1024):
        assert count(t, n, 20011, "bf16", k, False) == 0, k
    for k in (419, 420, 421, 512):
        ids = lp.top_logprobs(t, k)[0]
        assert torch.equal(ids, lp.top_logprobs(t, 513)[0][:, :k])
