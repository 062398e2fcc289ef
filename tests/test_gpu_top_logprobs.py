"""lp_top_logprobs against the fp64 oracle. Ids and logits are exact; logprobs
and lse are rounded to fp32 once (2^-24 relative) and have the error of the
token draw's raw score, derived there (86 * 2^-24 absolute, 2^-24 relative)."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import logit_rows as ol

from .gpu_helpers import DEV
from .logits_helpers import place, rows

pytestmark = pytest.mark.gpu


def check(t, z, k, temperature=1.0, v_true=None):
    lse = torch.full((z.shape[0],), float("nan"), device=DEV)
    got = lp.top_logprobs(t, k, temperature, v_true, lse=lse)
    torch.cuda.synchronize()
    ids, val, logp = (g.cpu().numpy() for g in got)
    r_ids, r_val, r_lp, r_lse = ol.top_logprobs(z, k, temperature)
    print("rows", z.shape, "k", k)
    assert np.array_equal(ids, r_ids)
    assert np.array_equal(val, r_val.astype(np.float32), equal_nan=True)
    for g, r in ((logp, r_lp), (lse.cpu().numpy(), r_lse)):
        finite = np.isfinite(r)
        assert np.array_equal(g[~finite], r[~finite].astype(np.float32), equal_nan=True)
        assert np.all(np.abs(g[finite] - r[finite]) <= 2.0 ** -23 * np.abs(r[finite]) + 86 * 2.0 ** -24)
    return got


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,v,k,pad,lead", [(1, 1, 1, 0, 0), (2, 3, 3, 1, 1), (5, 9, 4, 0, 3),
                                            (7, 255, 255, 0, 0), (9, 1000, 20, 24, 0),
                                            (4, 1025, 1024, 3, 5), (16, 5003, 100, 0, 1),
                                            (3, 50021, 1024, 3, 0)])
def test_sizes(dtype, n, v, k, pad, lead):
    t, z = rows(v + k, n, v, dtype, pad=pad, lead=lead)
    check(t, z, k, 1.0)
    check(t, z, k, 1.7)


@pytest.mark.parametrize("dtype,k", [("bf16", 64), ("fp32", 20), ("fp32", 1)])
def test_a_language_models_vocabulary(dtype, k):
    t, z = rows(5, 5, 151936, dtype)
    check(t, z, k)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("kind", ["equal", "narrow", "steps", "far"])
def test_ties_and_crowded_buckets(dtype, kind):
    rng = np.random.default_rng(4)
    n, v = 4, 30011
    z = {"equal": np.full((n, v), -2.0), "narrow": rng.normal(size=(n, v)) * 1e-3,
         "steps": np.floor(rng.normal(size=(n, v)) * 2) / 2,
         "far": rng.normal(size=(n, v)) - 500.0}[kind]
    if kind == "far":
        z[:, 100] = 600.0      # everything else is far below the maximum
    t, z = place(z, dtype)
    for k in (1, 2, 64, 1024):
        check(t, z, k)


def test_the_smallest_temperature():
    tau = 2.0 ** -126
    z = np.random.default_rng(12).normal(size=(4, 9001)) * 4 * tau
    t, z = place(z, "fp32")
    check(t, z, 50, tau)


def test_masks_and_rows_without_logits():
    t, z = rows(6, 6, 3000, "fp32", masked=0.9)
    z[0, 20:] = -np.inf        # fewer finite logits than k
    z[1] = -np.inf
    z[2, 5], z[3, 6] = np.nan, np.inf
    t, z = place(z, "fp32")
    check(t, z, 50)
    with pytest.raises(ValueError, match="3 row"):
        lp.top_logprobs(t, 5, check=True)


def test_v_true_alignment_and_batch_invariance():
    t, z = rows(8, 20, 7001, "bf16")
    t[:, 6500:] = 40.0
    ref = check(t, z[:, :6500], 33, v_true=6500)
    t2, _ = place(z, "bf16", pad=7, lead=3)
    got = lp.top_logprobs(t2, 33, v_true=6500)
    one = lp.top_logprobs(t2[11:12], 33, v_true=6500)
    for a, b, c in zip(ref, got, one):
        assert torch.equal(a, b) and torch.equal(a[11:12], c)


def test_wrong_arguments():
    z = torch.zeros(4, 10, device=DEV)
    for k in (0, 11, -1, 1025):
        with pytest.raises(ValueError):
            lp.top_logprobs(z, k)
    with pytest.raises(lp.LpError):
        lp.top_logprobs(z, 3, temperature=0.0)
    assert lp.top_logprobs(z[:0], 3)[0].shape == (0, 3)
