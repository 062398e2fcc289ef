"""The operators on rows of logits together with the rest of the library, as
an on-policy distillation step uses them; streams, and graphs that are
captured and replayed."""

import numpy as np
import pytest
import torch

import oracle
import rollout_logprob_consistency_amd as lp
from oracle import logit_rows as ol
from workloads import synth

from .gpu_helpers import DEV, SCORE_ATOL, dev_bf16
from .logits_helpers import TYPES

pytestmark = pytest.mark.gpu


def test_rollout_teacher_distillation_step():
    """Draw tokens from the student's logits; their raw scores agree with
    lp_score of the same hidden states; the teacher's top logits; the loss
    and its gradient at the student's hidden states."""
    c = synth.tiny_case(T=48, H=256, V=4096)
    x, w = dev_bf16(c.x_bits), dev_bf16(c.w_bits)
    g = torch.Generator(device=DEV).manual_seed(1)
    student = x.float() @ w.float().t()                       # fp32 logits of the LM head
    teacher_w = w.float() + 0.01 * torch.randn(w.shape, generator=g, device=DEV)
    teacher = x.float() @ teacher_w.t()
    u = torch.rand(48, generator=g, device=DEV)
    tau = 0.8
    token, raw, processed, kept = lp.sample(student, u, tau, 40, 0.9, check=True)
    z = student.double().cpu().numpy()
    ref = ol.sample(z, u.cpu().numpy(), tau, 40, 0.9)
    assert np.array_equal(token.cpu().numpy(), ref[0]) and np.array_equal(kept.cpu().numpy(), ref[3])
    assert (processed >= raw).all()
    # The raw score is lp_score's under the same temperature.
    score = lp.score(x, w, token, tau, check=True)
    assert (score - raw).abs().max().item() <= SCORE_ATOL
    o, _ = oracle.score(c.x_bits, c.w_bits, token.cpu().numpy(), tau)
    assert np.max(np.abs(o - raw.cpu().numpy())) <= SCORE_ATOL
    # Generation and replay scores of one sequence, compared.
    one = torch.ones(1, 48, dtype=torch.uint8, device=DEV)
    stats = lp.compare(raw[None], score[None], score[None], one)
    assert stats["AB"]["max_abs"][0] <= SCORE_ATOL and stats["BC"]["mismatch"][0] == 0

    ids, top, logp = lp.top_logprobs(teacher, 32, check=True)
    r_ids, r_top, r_logp, _ = ol.top_logprobs(teacher.double().cpu().numpy(), 32)
    assert np.array_equal(ids.cpu().numpy(), r_ids)
    hidden = x.float().clone().requires_grad_(True)
    logits = hidden @ w.float().t()
    weight = (torch.arange(48, device=DEV) >= 8).float() / 40      # eight prompt rows
    (lp.distill(logits, ids, top) * weight).sum().backward()
    loss, grad = ol.distill(z, r_ids, r_top, 1.0, True, weight.cpu().numpy())
    want = grad @ w.double().cpu().numpy()
    # The last product is torch's in fp32 over 4 096 terms; 1e-5 of the largest
    # value is 4 096^1/2 * 2^-24 with a factor of 3 to spare.
    assert np.max(np.abs(hidden.grad.double().cpu().numpy() - want)) <= 1e-5 * np.abs(want).max() + 1e-8
    # The teacher's logprobs as they are: a smaller weight per row, less loss mass.
    l2 = lp.distill(student, ids, logp, renormalize=False)
    assert torch.isfinite(l2).all()


@pytest.fixture(scope="module")
def batch():
    g = torch.Generator(device=DEV).manual_seed(2)
    z = torch.randn(24, 40001, generator=g, device=DEV) * 2.5
    u = torch.rand(24, generator=g, device=DEV)
    w = torch.rand(24, generator=g, device=DEV)
    ids, top, _ = lp.top_logprobs(z + 0.3, 50)
    torch.cuda.synchronize()
    return z, u, w, ids, top


def everything(z, u, w, ids, top):
    out = list(lp.sample(z, u, 0.9, 0, 0.9)) + list(lp.sample(z, u, 0.7, 30, 0.9))
    out += list(lp.top_logprobs(z, 64))
    loss, state = lp.distill_forward(z, ids, top)
    out += [loss, lp.distill_backward(z, ids, top, state, w)]
    out += list(lp.distill_step(z.bfloat16(), ids, top, w))
    return out


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_results_do_not_depend_on_the_batch(dtype):
    """520 rows (whole rows a workgroup) against single rows and batches of 40
    (rows cut into slices), with settings of every kind: short lists, lists
    that overflow (ties, many tokens above min-p), wide top-k, nuclei."""
    n, v = 520, 40009
    g = torch.Generator(device=DEV).manual_seed(4)
    z = torch.randn(n, v, generator=g, device=DEV) * 2.0
    z[::7] = (z[::7] * 2).round() / 2               # heavy ties
    z[::11, ::3] = float("-inf")
    z[5] = 1.25
    z[6, 77] = float("nan")
    z = z.to(TYPES[dtype])
    u = torch.rand(n, generator=g, device=DEV)

    def pick(options, kind):
        o = torch.tensor(options, dtype=kind, device=DEV)
        return o[torch.randint(0, len(options), (n,), generator=g, device=DEV)]
    how = (pick([0.0, 0.6, 1.0, 1.8], torch.float32), pick([0, 0, 1, 30, 400, 900], torch.int32),
           pick([1.0, 0.9, 0.5], torch.float32), pick([0.0, 0.0, 0.05, 1e-4], torch.float32))
    ref = lp.sample(z, u, *how)
    top = [lp.top_logprobs(z, k) for k in (20, 700)]
    spans = [slice(i, i + 1) for i in range(0, 40)] + [slice(i, i + 40) for i in range(40, 520, 40)]
    for s in spans:
        got = lp.sample(z[s], u[s], *(h[s] for h in how))
        for a, b in zip(ref, got):
            assert torch.equal(a[s].nan_to_num(-9), b.nan_to_num(-9)), s
        for k, t in zip((20, 700), top):
            for a, b in zip(t, lp.top_logprobs(z[s], k)):
                assert torch.equal(a[s].nan_to_num(-9), b.nan_to_num(-9)), (s, k)


def test_offsets_past_32_bits():
    """15 000 bf16 rows of 151 936 (2.3e9 logits, 4.6 GB): the last rows as they
    are alone, the gradient over the logits' own buffer."""
    n, v = 15000, 151936
    z = torch.zeros(n, v, dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(5)
    last = slice(n - 4, n)
    z[last] = torch.randn(4, v, generator=g, device=DEV).to(torch.bfloat16) * 3
    u = torch.rand(n, generator=g, device=DEV)
    w = torch.rand(n, generator=g, device=DEV)
    w[: n - 4] = 0
    alone = z[last].clone()
    for how in (dict(top_p=0.9), dict(top_k=30)):
        whole, one = lp.sample(z, u, **how), lp.sample(alone, u[last], **how)
        assert all(torch.equal(a[last], b) for a, b in zip(whole, one))
    whole, one = lp.top_logprobs(z, 16), lp.top_logprobs(alone, 16)
    assert all(torch.equal(a[last], b) for a, b in zip(whole, one))
    ids, top, _ = whole
    loss, grad = lp.distill_step(alone, ids[last].contiguous(), top[last].contiguous(), w[last])
    loss2, grad2 = lp.distill_step(z, ids, top, w, out=z)
    assert torch.equal(loss2[last], loss) and torch.equal(grad2[last], grad)
    assert not grad2[: n - 4].any()


def test_streams_give_the_default_streams_bits(batch):
    ref = everything(*batch)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(2):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(everything(*batch))
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(ref, out))


def test_graph_capture_and_replay(batch):
    """Captured once, replayed with other inputs in the same buffers and eager
    work in between; every replay equals the eager call."""
    z, u, w, ids, top = (t.clone() for t in batch)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        everything(z, u, w, ids, top)
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = everything(z, u, w, ids, top)
    torch.cuda.synchronize()
    for rep in range(3):
        z.add_(torch.randn_like(z) * 0.1)
        u.uniform_()
        want = everything(z, u, w, ids, top)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, out):
            assert torch.equal(a, b), rep


def test_a_step_captured_with_autograd(batch):
    """Loss and gradient through autograd inside a graph, no eager graph of the
    leaf alive; replays against the eager step."""
    z, _, w, ids, top = batch
    leaf = z.clone().requires_grad_(True)

    def step():
        loss = lp.distill(leaf, ids, top, 2.0)
        grad, = torch.autograd.grad(loss, leaf, w)
        return loss.detach(), grad

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=side):
            out = step()
    torch.cuda.synchronize()
    for rep in range(3):
        with torch.no_grad():
            leaf.add_(0.01 * rep)
        want = step()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out)), rep
