"""The scores of the token draw and the top logits where they are easily lost.

Tolerance where nothing else is said: the one derived in test_gpu_sample.py
(86 * 2^-24 absolute, 2^-23 relative)."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import logit_rows as ol

from .gpu_helpers import DEV
from .logits_helpers import dev, place

pytestmark = pytest.mark.gpu
F32 = torch.float32


def near(got, ref, tol):
    got = got.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref)), (got, ref)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), (got, ref)
    ok = np.isfinite(ref)
    err, tol = np.abs(got - ref, where=ok, out=np.zeros(ref.shape)), np.broadcast_to(tol, ref.shape)
    print("error / tolerance", np.max((err / tol)[ok], initial=0.0))
    assert np.all(err[ok] <= tol[ok]), (got[ok], ref[ok])


@pytest.mark.parametrize("n", [3, 530])
@pytest.mark.parametrize("scale,tau", [(3.0, 1e-4), (3.0, 1e-6), (3.0, 1e-8), (3.0, 3e-10),
                                       (1e6, 1.0), (1e9, 1.0), (3e10, 0.7), (1e11, 1.0), (1e12, 1.0)])
def test_large_quotients(n, scale, tau):
    """Logits over the temperature from 2^15 to 2^40: what a sum counts its
    exponents from is no longer a whole number of fp32 there."""
    rng = np.random.default_rng(n)
    v = 9001 if n == 3 else 700
    z = rng.normal(size=(n, v)) * scale
    z[1, 5:9] = z[1].max()                    # ties at the top
    z[2, 1:] = z[2, 0] * (1 - 2.0 ** -23 * rng.integers(0, 3, v - 1))
    t, z = place(z)
    u = rng.random(n, np.float32)
    for how in (dict(top_k=20), dict(min_p=0.05), dict(top_k=500, top_p=0.9), dict(top_p=0.9)):
        got = lp.sample(t, dev(u, F32), tau, **how)
        ref = ol.sample(z, u, tau, **how)
        assert np.array_equal(got[0].cpu().numpy(), ref[0])
        near(got[1], ref[1], 2.0 ** -23 * np.abs(ref[1]) + 86 * 2.0 ** -24)
    lse = torch.empty(n, device=DEV)
    ids, _, logp = lp.top_logprobs(t, 40, tau, lse=lse)
    r_ids, _, r_lp, r_lse = ol.top_logprobs(z, 40, tau)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    near(logp, r_lp, 2.0 ** -23 * np.abs(r_lp) + 86 * 2.0 ** -24)
    near(lse, r_lse, 2.0 ** -23 * np.abs(r_lse) + 86 * 2.0 ** -24)


def scores(z, tau, listed):
    """Per row: ln p of every token, the log-sum-exp, and the probability
    outside the `listed` first tokens of the order; each sum from its smallest
    term on, so that a confident row's small rest is not lost."""
    logp, lse, rest = np.empty(z.shape), np.empty(len(z)), np.empty(len(z))
    for i, row in enumerate(z):
        s = (row - row.max()) / tau
        w = np.sort(np.exp(s))
        below = w[:w.size - listed[i]].sum()
        others = w[:-1].sum()
        logp[i] = s - np.log1p(others)
        lse[i] = row.max() / tau + np.log1p(others)
        rest[i] = below / (1 + others)
    return logp, lse, rest


def tolerance(ref, rest):
    """The groups of the listed tokens are summed in fp64 (1e-13 and less in the
    sum). What is outside them has fp32 exponentials 2^(z c - b): one rounding
    of the exponent x, at most ln2 * 2^-24 |x| of a weight; c = log2 e / tau
    rounded, ln2 * 2^-24 |x| too; 2^-23 for the exponential, at most 7 additions
    of 2^-24. b is the integer next to the exponent of the largest logit among a
    wave's first groups: |x| of the largest weight outside is at most 126 (smaller ones
    weigh nothing), and weighted by the weights the others lie at most log2 V <=
    17.3 below it. (2 ln2 (126 + 17.3) + 9) * 2^-24 <= 210 * 2^-24 of `rest`.
    One rounding of the score to fp32."""
    return 2.0 ** -24 * np.abs(ref) + 210 * 2.0 ** -24 * rest + 1e-13


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,v", [(1, 151936), (8, 30011), (300, 9001), (40, 257)])
@pytest.mark.parametrize("gap", [0.0, 5.0, 12.0, 25.0])
def test_confident_rows(dtype, n, v, gap):
    """One token `gap` above the others: the score of a token that has nearly
    all of the probability is the little that the others have."""
    rng = np.random.default_rng(int(v + gap))
    z = rng.normal(size=(n, v)) * 2.2
    z[np.arange(n), rng.integers(0, v, n)] = z.max(1) + gap
    t, z = place(z, dtype)
    u = dev(rng.random(n, np.float32), F32)
    for tau in (1.0, 0.7, 1.3):
        tau = float(np.float32(tau))
        rows = np.arange(n)
        for how in (dict(top_k=20, top_p=0.95), dict(min_p=0.05), dict(greedy=True)):
            if "greedy" in how:
                token, raw, _, kept = lp.sample(t, u, 0.0)
                listed, at = np.full(n, 1), 1.0
            else:
                token, raw, _, kept = lp.sample(t, u, tau, **how)
                listed, at = np.full(n, 20) if "top_k" in how else kept.cpu().numpy(), tau
            logp, _, rest = scores(z, at, listed)
            ref = logp[rows, token.cpu().numpy()]
            near(raw, ref, tolerance(ref, rest))
            assert (raw <= 0).all()
        for k in (1, 20, min(v, 700)):
            lse = torch.empty(n, device=DEV)
            ids, _, got = lp.top_logprobs(t, k, tau, lse=lse)
            logp, r_lse, rest = scores(z, tau, np.full(n, k))
            ref = np.take_along_axis(logp, ids.cpu().numpy(), 1)
            near(got, ref, tolerance(ref, rest[:, None]))
            near(lse, r_lse, tolerance(r_lse, rest))


@pytest.mark.parametrize("n", [4, 300])
def test_confident_rows_whose_list_overflows(n):
    """More ties than a list holds, under tokens that have the probability."""
    v = 20011
    z = np.full((n, v), -30.0)
    rng = np.random.default_rng(1)
    for i in range(n):
        z[i, rng.integers(0, v, 3)] = [1.0, 0.5, -14.0]
    t, z = place(z)
    u = dev(rng.random(n, np.float32), F32)
    token, raw, _, _ = lp.sample(t, u, top_k=30)
    logp, _, rest = scores(z, 1.0, np.full(n, 30))
    ref = logp[np.arange(n), token.cpu().numpy()]
    near(raw, ref, tolerance(ref, rest))
    ids, _, got = lp.top_logprobs(t, 30)
    ref = np.take_along_axis(logp, ids.cpu().numpy(), 1)
    near(got, ref, tolerance(ref, rest[:, None]))
