"""The operators on rows of logits at the C boundary and in the binding:
declared and exported functions, and the refusals, which all come before
anything touches a device (CPU only)."""

import os
import re
import subprocess

import pytest
import torch

import rollout_logprob_consistency_amd as lp
from rollout_logprob_consistency_amd import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "liblp_logits.h")
EINVAL, EUNSUP = 1, 2
NAN, INF = float("nan"), float("inf")
P = 0x10000          # aligned, never dereferenced: every call below is refused
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def test_header_exports_and_constants(L):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = set(re.findall(r"\b(lp_[a-z_]+)\s*\(", text))
    assert declared == set(_lib.LOGITS_EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", _lib.LIB_PATH],
                         capture_output=True, text=True, check=True).stdout
    assert declared <= set(re.findall(r"\bT (lp_\w+)", out))
    for name, value in (("LP_SELECT_MAX_VOCAB", _lib.SELECT_MAX_VOCAB),
                        ("LP_TOP_MAX", _lib.TOP_MAX), ("LP_DISTILL_MAX_K", _lib.DISTILL_MAX_K),
                        ("LP_DISTILL_LOGPROBS", _lib.DISTILL_LOGPROBS),
                        ("LP_F32", 0), ("LP_BF16", 1), ("LP_F16", 2)):
        assert int(re.search(r"#define %s (\d+)" % name, open(HEADER).read()).group(1)) == value


def sample(L, logits=P, ld=100, dtype=0, N=4, V=100, u=P, ts=None, t=1.0, ks=None, k=0, ps=None,
           p=1.0, ms=None, m=0.0, tok=P, out=P, proc=None, kept=None, bad=None, ws=P, wsb=BIG):
    return L.lp_sample(logits, ld, dtype, N, V, u, ts, t, ks, k, ps, p, ms, m, tok, out, proc, kept,
                       bad, ws, wsb, None)


def test_sample_refusals(L):
    for kw in (dict(N=-1), dict(V=0), dict(ld=99), dict(dtype=3), dict(dtype=-1), dict(t=-0.5),
               dict(t=NAN), dict(t=INF), dict(p=NAN), dict(m=NAN), dict(logits=None), dict(u=None),
               dict(tok=None), dict(out=None), dict(ws=None), dict(logits=P + 2),
               dict(logits=P + 1, dtype=1), dict(u=P + 2), dict(ts=P + 1), dict(ks=P + 2),
               dict(ps=P + 2), dict(ms=P + 2), dict(tok=P + 4), dict(out=P + 2), dict(proc=P + 2),
               dict(kept=P + 2), dict(bad=P + 2), dict(ws=P + 16), dict(wsb=0)):
        assert sample(L, **kw) == EINVAL, kw
    big = _lib.SELECT_MAX_VOCAB + 1
    assert sample(L, V=big, ld=big) == EUNSUP
    assert sample(L, N=4194304) == EUNSUP
    assert sample(L, N=0, logits=None, u=None, tok=None, out=None, ws=None) == 0


def top(L, logits=P, ld=100, dtype=0, N=4, V=100, k=5, t=1.0, ids=P, z=P, out=P, lse=None, bad=None,
        ws=P, wsb=BIG):
    return L.lp_top_logprobs(logits, ld, dtype, N, V, k, t, ids, z, out, lse, bad, ws, wsb, None)


def test_top_refusals(L):
    for kw in (dict(N=-1), dict(V=0), dict(ld=99), dict(dtype=7), dict(k=0), dict(k=101),
               dict(t=0.0), dict(t=-1.0), dict(t=NAN), dict(t=INF), dict(logits=None),
               dict(ids=None), dict(z=None), dict(out=None), dict(ws=None), dict(logits=P + 2),
               dict(ids=P + 4), dict(z=P + 2), dict(out=P + 1), dict(lse=P + 2), dict(bad=P + 2),
               dict(ws=P + 128), dict(wsb=0)):
        assert top(L, **kw) == EINVAL, kw
    assert top(L, k=1025, V=2000, ld=2000) == EUNSUP
    big = _lib.SELECT_MAX_VOCAB + 1
    assert top(L, V=big, ld=big) == EUNSUP
    assert top(L, N=4194304) == EUNSUP
    assert top(L, N=0, logits=None, ids=None, z=None, out=None, ws=None) == 0


def forward(L, logits=P, ld=100, dtype=0, T=4, V=100, ids=P, x=P, K=5, t=1.0, flags=0, loss=P,
            state=P, bad=None, ws=P, wsb=BIG):
    return L.lp_distill_forward(logits, ld, dtype, T, V, ids, x, K, t, flags, loss, state, bad, ws,
                                wsb, None)


def backward(L, logits=P, ld=100, dtype=0, T=4, V=90, C=100, ids=P, x=P, K=5, t=1.0, flags=0,
             state=P, g=P, out=P, ldg=100):
    return L.lp_distill_backward(logits, ld, dtype, T, V, C, ids, x, K, t, flags, state, g, out,
                                 ldg, None)


def step(L, logits=P, ld=100, dtype=0, T=4, V=90, C=100, ids=P, x=P, K=5, t=1.0, flags=0, w=P,
         loss=P, out=P, ldg=100, bad=None, ws=P, wsb=BIG):
    return L.lp_distill_step(logits, ld, dtype, T, V, C, ids, x, K, t, flags, w, loss, out, ldg,
                             bad, ws, wsb, None)


def test_distill_refusals(L):
    for call in (forward, backward, step):
        for kw in (dict(T=-1), dict(V=0), dict(ld=89), dict(K=0), dict(dtype=3), dict(flags=2),
                   dict(t=0.0), dict(t=NAN), dict(t=INF), dict(logits=None), dict(ids=None),
                   dict(x=None), dict(logits=P + 2), dict(ids=P + 4), dict(x=P + 2)):
            assert call(L, **kw) == EINVAL, (call, kw)
        assert call(L, K=1025) == EUNSUP
        assert call(L, T=1 << 31) == EUNSUP
    for kw in (dict(loss=None), dict(loss=P + 2), dict(state=P + 4), dict(bad=P + 2),
               dict(ws=None), dict(ws=P + 8), dict(wsb=16)):
        assert forward(L, **kw) == EINVAL, kw
    assert forward(L, V=1 << 31, ld=1 << 31) == EUNSUP
    for kw in (dict(C=89), dict(ldg=99), dict(state=None), dict(g=None), dict(out=None),
               dict(state=P + 4), dict(g=P + 2), dict(out=P + 2)):
        assert backward(L, **kw) == EINVAL, kw
    for kw in (dict(C=89), dict(ldg=99), dict(w=None), dict(loss=None), dict(out=None),
               dict(w=P + 2), dict(out=P + 2), dict(bad=P + 2), dict(ws=None), dict(wsb=16)):
        assert step(L, **kw) == EINVAL, kw
    assert forward(L, T=0, logits=None, ids=None, x=None, loss=None, ws=None) == 0
    assert backward(L, T=0, logits=None, ids=None, x=None, state=None, g=None, out=None) == 0
    assert step(L, T=0, logits=None, ids=None, x=None, w=None, loss=None, out=None, ws=None) == 0


def test_workspace_bytes(L):
    for f in (L.lp_sample_workspace_bytes, L.lp_top_logprobs_workspace_bytes,
              L.lp_distill_workspace_bytes):
        assert f(-1, 100, 0) == 0 and f(4, 0, 0) == 0 and f(4, 100, 3) == 0
        assert f(0, 100, 0) > 0 and f(4, 100, 1) % 256 == 0
    # distillation: a maximum and a sum per slice of at most 16 KiB x 2, 32 bytes a row
    assert L.lp_distill_workspace_bytes(8192, 151936, 1) >= 8192 * (10 * 12 + 32)


def test_binding_refuses_what_it_cannot_pass_on():
    z, u = torch.zeros(4, 10), torch.zeros(4)
    ids, x = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2)
    for call in (lambda: lp.sample(z, u), lambda: lp.top_logprobs(z, 2),
                 lambda: lp.distill(z, ids, x), lambda: lp.distill_forward(z, ids, x),
                 lambda: lp.distill_step(z, ids, x, u)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
    with pytest.raises(ValueError, match="must not require gradients"):
        lp.distill(z, ids, x.clone().requires_grad_(True))


@pytest.mark.parametrize("t", [2.0 ** -127, 1e-45, -1e-45])
def test_subnormal_temperatures_are_refused(L, t):
    for call in (sample, top, forward, backward, step):
        assert call(L, t=t) == EINVAL, call


@pytest.mark.parametrize("dtype", [0, 1, 2])
@pytest.mark.parametrize("V", [1, 1025, 9001, 151936, _lib.SELECT_MAX_VOCAB])
def test_a_workspace_serves_fewer_rows_and_smaller_vocabularies(L, dtype, V):
    """Sizes ascend with the rows and with the vocabulary: a caller's buffer for
    its largest batch is not refused for a smaller one."""
    rows = list(range(0, 700)) + [1000, 4096, 100000, 4194303]
    for f in (L.lp_sample_workspace_bytes, L.lp_top_logprobs_workspace_bytes,
              L.lp_distill_workspace_bytes):
        sizes = [f(n, V, dtype) for n in rows]
        assert sizes == sorted(sizes) and all(s % 256 == 0 for s in sizes)
        for n in (1, 5, 39, 256, 257, 512, 513, 4096):
            by_v = [f(n, v, dtype) for v in (1, 300, 4096, 4097, 8193, 30000, 151936, 1048576)]
            assert by_v == sorted(by_v)
    # Scratch memory stays within tens of megabytes, but for a row's counter.
    assert L.lp_sample_workspace_bytes(4096, V, dtype) < 40 << 20
