"""Temperatures whose inverse fp32 cannot hold, at every scoring entry point (CPU
only: the calls have no rows, so that those that are accepted do nothing)."""

import pytest

from rollout_logprob_consistency_amd import _lib

EINVAL = 1
P = 0x10000          # aligned, never dereferenced
LEAST = 4.24e-39     # log2(e) over it is just below fp32's largest number


@pytest.fixture(scope="module")
def calls():
    L = _lib.lib()
    return {
        "lp_score": lambda t: L.lp_score(P, 64, P, P, 0, 64, 300, 300, t, P, None, None, P, 1 << 30,
                                         None),
        "lp_score_stats": lambda t: L.lp_score_stats(P, 64, P, P, 0, 64, 300, 300, t, P, None, P, P,
                                                     None, P, 1 << 30, None),
        "lp_score_ex": lambda t: L.lp_score_ex(P, 64, P, P, 0, 64, 300, 300, t, 2, P, None, None,
                                               None, None, P, 1 << 30, None),
        "lp_score_noalloc": lambda t: L.lp_score_noalloc(P, 64, P, P, 0, 64, 300, 300, t, P, None,
                                                         None, None),
        "lp_score_shard": lambda t: L.lp_score_shard(P, 64, P, P, 0, 64, 300, t, 2, 0, 0, P, P,
                                                     1 << 30, None),
    }


@pytest.mark.parametrize("t", [4.239e-39, 1e-39, 1e-45, 0.0, -1e-39, -1.0, float("inf"),
                               float("nan")])
def test_refused(calls, t):
    for name, call in calls.items():
        assert call(t) == EINVAL, name


@pytest.mark.parametrize("t", [LEAST, 2.0 ** -127, 2.0 ** -126, 1e-3, 1.0, 3e38])
def test_accepted(calls, t):
    for name, call in calls.items():
        assert call(t) == 0, name
