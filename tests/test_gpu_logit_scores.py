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
