"""The 8-bit head at the C boundary and in the binding: declared and exported
functions, and the refusals, which all come before anything touches a device
(CPU only)."""

import os
import re
import subprocess

import pytest
import torch

import rollout_logprob_consistency_amd as lp
from rollout_logprob_consistency_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "liblp_int8.h")
EINVAL, EUNSUP = 1, 2
NAN, INF = float("nan"), float("inf")
P = 0x10000          # aligned, never dereferenced: every call below is refused
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_header_exports_and_constants():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(lp_[a-z0-9_]+)\s*\(", text))
    assert declared == set(_lib.INT8_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH],
                         capture_output=True, text=True, check=True).stdout
    assert declared <= set(re.findall(r"\bT (lp_\w+)", out))
    most = re.search(r"#define LP_INT8_MAX_HIDDEN (\d+)", open(HEADER).read()).group(1)
    assert int(most) == _lib.INT8_MAX_HIDDEN
    assert _lib.INT8_MAX_HIDDEN * 2 ** 14 < 2 ** 31 <= (_lib.INT8_MAX_HIDDEN + 1) * 2 ** 14


def quantize(L, x=P, ldx=100, dtype=0, R=4, H=100, q=P, ldq=112, scale=P, bad=None):
    return L.lp_quantize_int8(x, ldx, dtype, R, H, q, ldq, scale, bad, None)


def test_quantize_refusals(L):
    for kw in (dict(R=-1), dict(H=0), dict(ldx=99), dict(ldq=96), dict(ldq=104), dict(dtype=3),
               dict(dtype=-1), dict(x=None), dict(q=None), dict(scale=None), dict(x=P + 2),
               dict(x=P + 1, dtype=1), dict(q=P + 8), dict(scale=P + 2), dict(bad=P + 2)):
        assert quantize(L, **kw) == EINVAL, kw
    assert quantize(L, R=16777216) == EUNSUP
    assert quantize(L, H=2 ** 31, ldx=2 ** 31, ldq=2 ** 31) == EUNSUP
    assert quantize(L, R=0, x=None, q=None, scale=None) == 0


def logits(L, x=P, ldx=100, xs=P, w=P, ldw=112, ws=P, T=4, H=100, V=50, out=P, ldo=50, dtype=0,
           wk=P, wkb=BIG):
    return L.lp_logits_int8(x, ldx, xs, w, ldw, ws, T, H, V, out, ldo, dtype, wk, wkb, None)


def score(L, x=P, ldx=100, xs=P, w=P, ldw=112, ws=P, ids=P, T=4, H=100, V=50, t=1.0, flags=0,
          out=P, lse=None, bad=None, wk=P, wkb=BIG):
    return L.lp_score_int8(x, ldx, xs, w, ldw, ws, ids, T, H, V, t, flags, out, lse, bad, wk, wkb,
                           None)


SHARED = (dict(T=-1), dict(H=0), dict(V=0), dict(ldx=99), dict(ldw=96), dict(x=None),
          dict(xs=None), dict(w=None), dict(ws=None), dict(w=P + 8), dict(xs=P + 2),
          dict(ws=P + 1), dict(out=None), dict(wk=None), dict(wk=P + 128), dict(wkb=0))


def test_logits_refusals(L):
    for kw in SHARED + (dict(ldo=49), dict(dtype=5), dict(out=P + 2), dict(out=P + 1, dtype=2)):
        assert logits(L, **kw) == EINVAL, kw
    for kw in (dict(ldw=104), dict(ldw=2 ** 22 + 16), dict(ldo=2 ** 22 + 1), dict(H=131072, ldx=131072, ldw=131072),
               dict(T=4194241), dict(V=2 ** 31 - 255, ldo=2 ** 31),
               dict(T=100000, V=10 ** 7, ldo=10 ** 7)):
        assert logits(L, **kw) == EUNSUP, kw
    assert logits(L, T=0, x=None, xs=None, w=None, ws=None, out=None, wk=None) == 0


def test_score_refusals(L):
    for kw in SHARED + (dict(t=0.0), dict(t=-1.0), dict(t=NAN), dict(t=INF), dict(flags=1),
                        dict(flags=4), dict(ids=None), dict(ids=P + 4), dict(out=P + 2),
                        dict(lse=P + 1), dict(bad=P + 2)):
        assert score(L, **kw) == EINVAL, kw
    for kw in (dict(ldw=104), dict(H=131072, ldx=131072, ldw=131072), dict(T=4194241),
               dict(V=2 ** 31 - 255)):
        assert score(L, **kw) == EUNSUP, kw
    assert score(L, T=0, x=None, xs=None, w=None, ws=None, ids=None, out=None, wk=None) == 0


def test_workspaces(L):
    assert L.lp_logits_int8_workspace_bytes(4, 100) >= 4 * 128
    assert L.lp_logits_int8_workspace_bytes(0, 1) >= 1
    assert L.lp_score_int8_workspace_bytes(4, 100, 1000) >= 4 * 128 + 2 * 8 * 4 * 4
    for args in ((-1, 10), (2 ** 31, 10), (4, 0), (4, 131072)):
        assert L.lp_logits_int8_workspace_bytes(*args) == 0
        assert L.lp_score_int8_workspace_bytes(*args, 100) == 0
    assert L.lp_score_int8_workspace_bytes(4, 10, 0) == 0
    assert L.lp_score_int8_workspace_bytes(4, 10, 2 ** 31 - 255) == 0


def test_the_binding_refuses_what_does_not_lie_on_a_device():
    x = torch.zeros(2, 32, dtype=torch.int8)
    s = torch.ones(2)
    with pytest.raises(ValueError, match="CUDA"):
        lp.quantize_int8(torch.zeros(2, 32))
    with pytest.raises(ValueError, match="CUDA"):
        lp.logits_int8(x, s, x, s)
    with pytest.raises(ValueError, match="CUDA"):
        lp.score_int8(x, s, x, s, torch.zeros(2, dtype=torch.int64))
