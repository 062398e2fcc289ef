"""Calls of the operators on rows of logits that their documentation allows
beside the plain ones: counters and scratch memory of the caller's."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp

from .gpu_helpers import DEV
from .logits_helpers import rows

pytestmark = pytest.mark.gpu


def test_checked_calls_with_a_counter_that_is_not_zero():
    t, _ = rows(4, 6, 700)
    wrong = t.clone()
    wrong[2, 5] = wrong[4, 6] = float("nan")
    u = torch.full((6,), 0.5, device=DEV)
    ids = torch.zeros(6, 3, dtype=torch.int64, device=DEV)
    outside = ids.clone()
    outside[1, 2] = outside[5, 0] = 700
    x, w = torch.zeros(6, 3, device=DEV), torch.ones(6, device=DEV)
    calls = [(lambda bad, z: lp.sample(z, u, top_k=5, bad_rows=bad, check=True), t, wrong),
             (lambda bad, z: lp.sample(z, u, top_p=0.9, bad_rows=bad, check=True), t, wrong),
             (lambda bad, z: lp.top_logprobs(z, 5, bad_rows=bad, check=True), t, wrong),
             (lambda bad, i: lp.distill_forward(t, i, x, bad_rows=bad, check=True), ids, outside),
             (lambda bad, i: lp.distill_step(t, i, x, w, bad_rows=bad, check=True), ids, outside)]
    for call, clean, broken in calls:
        bad = torch.full((1,), 3, dtype=torch.int32, device=DEV)
        call(bad, clean)
        assert bad.item() == 3
        with pytest.raises(ValueError, match="^2 row"):
            call(bad, broken)
        assert bad.item() == 5
    bad = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    lp.sample(wrong, u, top_k=5, bad_rows=bad)
    lp.top_logprobs(wrong, 5, bad_rows=bad)
    assert bad.item() == 7


def workspace(need, tail=4096):
    """Scratch memory of exactly `need` bytes with something in it, and what lies behind."""
    buf = torch.full((need + tail,), 0xFF, dtype=torch.uint8, device=DEV)
    assert buf.data_ptr() % 256 == 0
    return buf[:need], buf[need:]


def batch(n, v, dtype, seed=5):
    t, z = rows(seed, n, v, dtype)
    z[0, : v // 2] = 3.0          # ties: a list that overflows
    t[0, : v // 2] = 3.0
    g = torch.Generator(device=DEV).manual_seed(seed)
    u = torch.rand(n, generator=g, device=DEV)
    w = torch.rand(n, generator=g, device=DEV)
    ids = torch.randint(0, v, (n, 20), generator=g, device=DEV)
    x = torch.randn(n, 20, generator=g, device=DEV)
    calls = {
        "lp_sample_workspace_bytes": [lambda s, **k: lp.sample(t[s], u[s], top_k=30, **k),
                                      lambda s, **k: lp.sample(t[s], u[s], 0.7, top_p=0.9, **k),
                                      lambda s, **k: lp.sample(t[s], u[s], min_p=0.01, **k)],
        "lp_top_logprobs_workspace_bytes": [lambda s, **k: lp.top_logprobs(t[s], 20, **k),
                                            lambda s, **k: lp.top_logprobs(t[s], 800, **k)],
        "lp_distill_workspace_bytes": [
            lambda s, **k: lp.distill_forward(t[s], ids[s], x[s], **k),
            lambda s, **k: lp.distill_step(t[s], ids[s], x[s], w[s], **k)],
    }
    return t, calls


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("n,v", [(1, 900), (3, 40009), (40, 20011), (300, 9001)])
def test_a_workspace_of_exactly_the_size(dtype, n, v):
    """Its contents on entry are ignored, what lies behind it is left alone, and
    it serves one call after another, of fewer rows too."""
    t, calls = batch(n, v, dtype)
    code = {"fp32": 0, "bf16": 1}[dtype]
    for name, fns in calls.items():
        ws, tail = workspace(getattr(lp.lib(), name)(n, v, code))
        for m in sorted({n, (n + 1) // 2, 1}, reverse=True):
            for call in fns:
                s = slice(n - m, n)
                print(name, n, m, flush=True)
                want, got = call(s), call(s, workspace=ws)
                for a, b in zip(want, got):
                    assert torch.equal(a.nan_to_num(-9), b.nan_to_num(-9)), (name, m)
                assert (tail == 0xFF).all()


def test_a_workspace_that_is_too_small():
    t, calls = batch(3, 40009, "fp32")
    for name, fns in calls.items():
        need = getattr(lp.lib(), name)(3, 40009, 0)
        for call in fns:
            with pytest.raises(lp.LpError):
                call(slice(0, 3), workspace=torch.empty(need - 256, dtype=torch.uint8, device=DEV))


def test_the_largest_batchs_workspace_serves_a_captured_smaller_one():
    """Buffers for 600 rows, a graph of 5 of them, replayed beside eager calls."""
    t, calls = batch(600, 20011, "bf16")
    ws, tail = workspace(lp.lib().lp_sample_workspace_bytes(600, 20011, 1))
    call, s = calls["lp_sample_workspace_bytes"][0], slice(0, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call(s, workspace=ws)
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = call(s, workspace=ws)
    torch.cuda.synchronize()
    for rep in range(3):
        t.add_(torch.randn_like(t) * 0.1)
        want = call(s)
        call(slice(0, 600), workspace=ws)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), rep
    assert (tail == 0xFF).all()
