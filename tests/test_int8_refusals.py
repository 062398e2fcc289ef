"""Calls of the 8-bit head that are refused, or are not, by what their arguments
say (CPU only: nothing here reaches a device)."""

import pytest

from rollout_logprob_consistency_amd import _lib

EINVAL, EUNSUP = 1, 2
P = 0x10000          # aligned, never dereferenced: every call below is refused
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def score(L, x=P, ldx=100, xs=P, w=P, ldw=112, ws=P, ids=P, T=4, H=100, V=50, t=1.0, flags=0,
          out=P, lse=None, bad=None, wk=P, wkb=BIG):
    return L.lp_score_int8(x, ldx, xs, w, ldw, ws, ids, T, H, V, t, flags, out, lse, bad, wk, wkb,
                           None)


@pytest.mark.parametrize("t", [2.0 ** -127, 1e-39, 1e-45, -1e-45])
def test_subnormal_temperatures_are_refused(L, t):
    """Their fp32 scale would be infinite, and every score NaN."""
    for flags in (0, 2):
        assert score(L, t=t, flags=flags) == EINVAL


def test_sizes_that_the_kernels_take(L):
    """A call passes the checks of its sizes if it gets as far as its workspace. The tile
    kernel is persistent: how many tiles there are is no matter of the dispatch."""
    for T, V in ((905000, 151936), (4194240, 151936), (4194240, 1 << 20), (33, 2 ** 31 - 256)):
        assert score(L, T=T, V=V, wkb=0) == EINVAL
    # More tiles than 32 bits count.
    for T, V in ((4194240, 2 ** 25), (65281, 2 ** 31 - 256)):
        assert score(L, T=T, V=V) == EUNSUP
    assert score(L, T=4194241) == EUNSUP
