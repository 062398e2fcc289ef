"""Verification of drafted tokens at the C boundary: the refusals, which all
come before anything touches a device (CPU only)."""

import re
import os

import pytest
import torch

import rollout_logprob_consistency_amd as lp
from rollout_logprob_consistency_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EINVAL, EUNSUP = 1, 2
NAN, INF = float("nan"), float("inf")
P = 0x10000          # aligned, never dereferenced: every call below is refused
BIG = 1 << 50


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def verify(L, logits=P, ld=100, dtype=0, B=4, D=3, V=100, draft=None, ldd=0, ids=P, counts=None,
           u=P, ts=None, t=1.0, ks=None, k=0, ps=None, p=1.0, ms=None, m=0.0, tok=P, acc=P, out=P,
           proc=None, bad=None, ws=P, wsb=BIG):
    return L.lp_verify(logits, ld, dtype, B, D, V, draft, ldd, ids, counts, u, ts, t, ks, k, ps, p,
                       ms, m, tok, acc, out, proc, bad, ws, wsb, None)


def test_verify_refusals(L):
    for kw in (dict(B=-1), dict(D=-1), dict(V=0), dict(ld=99), dict(draft=P, ldd=99),
               dict(dtype=3), dict(t=-0.5), dict(t=NAN), dict(t=INF), dict(p=NAN), dict(m=NAN),
               dict(logits=None), dict(ids=None), dict(u=None), dict(tok=None), dict(acc=None),
               dict(out=None), dict(ws=None), dict(logits=P + 2), dict(logits=P + 1, dtype=1),
               dict(draft=P + 1, ldd=100), dict(ids=P + 4), dict(counts=P + 2), dict(u=P + 2),
               dict(ts=P + 1), dict(ks=P + 2), dict(ps=P + 2), dict(ms=P + 2), dict(tok=P + 4),
               dict(acc=P + 2), dict(out=P + 2), dict(proc=P + 1), dict(bad=P + 2),
               dict(ws=P + 128), dict(wsb=0)):
        assert verify(L, **kw) == EINVAL, kw
    big = _lib.SELECT_MAX_VOCAB + 1
    for kw in (dict(D=64), dict(V=big, ld=big), dict(B=599187, D=3)):
        assert verify(L, **kw) == EUNSUP, kw
    assert verify(L, B=0, logits=None, ids=None, u=None, tok=None, acc=None, out=None, ws=None) == 0


def test_workspaces(L):
    size = L.lp_verify_workspace_bytes
    assert size(4, 3, 1000, 0) >= 4 * 7 * 32 + 4 * 8
    assert size(0, 0, 1, 0) > 0
    for b, d, v in ((3, 4, 5000), (64, 4, 151936), (600, 1, 20000)):
        most = size(b, d, v, 1)
        assert all(size(bb, dd, vv, 1) <= most
                   for bb in (1, b // 2 + 1, b) for dd in (0, 1, d) for vv in (1, v // 3, v))
    for args in ((-1, 3, 100, 0), (4, -1, 100, 0), (4, 64, 100, 0), (4, 3, 0, 0), (4, 3, 100, 3),
                 (4, 3, _lib.SELECT_MAX_VOCAB + 1, 0), (599187, 3, 100, 0)):
        assert size(*args) == 0
    text = open(os.path.join(ROOT, "include", "liblp_logits.h")).read()
    most = re.search(r"#define LP_VERIFY_MAX_DRAFTS (\d+)", text).group(1)
    assert int(most) == _lib.VERIFY_MAX_DRAFTS


def test_the_binding_refuses_what_does_not_lie_on_a_device():
    with pytest.raises(ValueError, match="CUDA"):
        lp.verify(torch.zeros(4, 10), torch.zeros(2, 1, dtype=torch.int64), torch.zeros(2, 2))
