"""Speculative decoding on an 8-bit head as an engine runs it, its calls on other
streams and in captured graphs, and offsets past 32 bits."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import int8_head, logit_rows
from oracle import verify as oracle_verify
from rollout_logprob_consistency_amd._lib import lib
from workloads import synth

from .gpu_helpers import DEV, dev_bf16

pytestmark = pytest.mark.gpu

B, D = 24, 3


def engine(seed=3):
    """Hidden states of B sequences at D + 1 positions, a head, and a draft that
    sees the same states through a noisier head."""
    c = synth.tiny_case(T=B * (D + 1), H=256, V=4096, seed=seed)
    x, w = dev_bf16(c.x_bits), dev_bf16(c.w_bits)
    g = torch.Generator(device=DEV).manual_seed(seed)
    draft_w = (w.float() + 0.02 * torch.randn(w.shape, generator=g, device=DEV)).bfloat16()
    u = torch.rand(B, D + 1, generator=g, device=DEV)
    return x, w, draft_w, u, torch.rand(B * D, generator=g, device=DEV)


def decode(x, head, draft_head, u, u_draft, how):
    """One step: the draft's tokens, the target's rows, the verdict. (Hidden
    states are given for every position, so the draft needs no loop.)"""
    q, s = lp.quantize_int8(x)
    at = torch.arange(B * (D + 1), device=DEV).view(B, D + 1)[:, :D].flatten()
    draft = lp.logits_int8(q[at], s[at], *draft_head)
    ids = lp.sample(draft, u_draft, **how)[0].view(B, D)
    target = lp.logits_int8(q, s, *head)
    return (q, s, draft, ids, target) + lp.verify(target, ids, u, draft, **how)


@pytest.mark.parametrize("how", [dict(temperature=0.7), dict(temperature=1.0, top_k=30, top_p=0.9),
                                 dict(top_p=0.8), dict(temperature=0.0)], ids=str)
def test_an_engines_step_and_its_scores(how):
    x, w, draft_w, u, u_draft = engine()
    head, draft_head = lp.quantize_int8(w), lp.quantize_int8(draft_w)
    q, s, draft, ids, target, tokens, accepted, raw, proc = decode(x, head, draft_head, u, u_draft,
                                                                    how)
    # Each step is the oracle's of what the one before gave.
    z = torch.from_numpy(int8_head.logits_f32(q.cpu(), s.cpu(), head[0].cpu(), head[1].cpu()))
    assert torch.equal(target.cpu().view(torch.int16), z.bfloat16().view(torch.int16))
    exact, exact_draft = target.double().cpu().numpy(), draft.double().cpu().numpy()
    want = logit_rows.sample(exact_draft, u_draft.cpu().numpy(), **how)
    assert np.array_equal(ids.cpu().numpy().ravel(), want[0])
    want = oracle_verify.verify(exact, ids.cpu().numpy(), u.cpu().numpy(), exact_draft, **how)
    assert np.array_equal(tokens.cpu().numpy(), want[0])
    assert np.array_equal(accepted.cpu().numpy(), want[1])
    assert 0 < accepted.sum() < B * D
    # The emitted tokens scored as the engine's bf16 logits have them are the raw
    # scores that the verdict came with (fp32 sums of 4 096 exponentials: 1e-5).
    tau = how.get("temperature", 1.0) or 1.0
    there = tokens >= 0
    scored = lp.score_int8(q, s, *head, tokens.clamp(min=0).flatten(), tau, bf16_logits=True,
                           check=True).view(B, D + 1)
    assert (scored - raw)[there].abs().max() <= 2e-5 * (1 + raw[there].abs().max())
    assert (proc >= raw - 1e-6)[there].all()
    # And the trainer's bf16 head scores them near: what quantisation changes.
    trained = lp.score(x, w, tokens.clamp(min=0).flatten(), tau, check=True).view(B, D + 1)
    gap = (trained - scored)[there].abs()
    assert 0 < gap.max() < 1.0
    mask = there.to(torch.uint8)
    stats = lp.compare(raw, scored, trained, mask)
    assert (stats["AB"]["max_abs"] <= 2e-5 * (1 + raw.abs().max().item())).all()


def outputs(t):
    return [x.contiguous().view(torch.uint8).clone() for x in t]


def test_other_streams_give_the_default_streams_bits():
    x, w, draft_w, u, u_draft = engine()
    head, draft_head = lp.quantize_int8(w), lp.quantize_int8(draft_w)
    how = dict(temperature=0.8, top_p=0.95)
    ref = outputs(decode(x, head, draft_head, u, u_draft, how))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for rep in range(2):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(decode(x, head, draft_head, u, u_draft, how))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(outputs(g), ref))


@pytest.mark.parametrize("rows", [2, 24, 300])
def test_a_captured_step_replays(rows):
    """The quantiser, both products and the verdict in one graph, replayed on new
    inputs in the same buffers, with eager work between the replays."""
    h, v, d = 320, 3001, 2
    g = torch.Generator(device=DEV).manual_seed(rows)
    head = lp.quantize_int8(torch.randn(v, h, generator=g, device=DEV))
    n = rows * (d + 1)
    x = torch.empty(n, h, dtype=torch.bfloat16, device=DEV)
    ids = torch.zeros(rows, d, dtype=torch.int64, device=DEV)
    u = torch.empty(rows, d + 1, device=DEV)
    q = torch.empty(n, h, dtype=torch.int8, device=DEV)
    s = torch.empty(n, device=DEV)
    z = torch.empty(n, v, dtype=torch.bfloat16, device=DEV)
    scores = torch.empty(n, device=DEV)
    ws = [torch.empty(max(size, 1), dtype=torch.uint8, device=DEV) for size in (
        lib().lp_logits_int8_workspace_bytes(n, h), lib().lp_score_int8_workspace_bytes(n, h, v),
        lib().lp_verify_workspace_bytes(rows, d, v, 1))]
    targets = torch.arange(n, device=DEV) % v

    def fill(seed):
        g.manual_seed(seed)
        x.normal_(generator=g)
        u.uniform_(generator=g)
        ids.random_(0, v, generator=g)

    def step():
        lp.quantize_int8(x, out=q, scale=s)
        lp.logits_int8(q, s, *head, out=z, workspace=ws[0])
        lp.score_int8(q, s, *head, targets, out=scores, workspace=ws[1])
        return lp.verify(z, ids, u, temperature=0.9, top_p=0.9, workspace=ws[2])

    fill(0)
    step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            held = step()
    for seed in (1, 2, 3):
        fill(seed)
        eager = outputs(list(step()) + [q, s, z, scores])
        for t in (q, s, z, scores, *held, *ws):
            t.fill_(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = outputs(list(held) + [q, s, z, scores])
        assert all(torch.equal(a, b) for a, b in zip(got, eager)), seed
        torch.randn(1 << 20, device=DEV).sum().item()


# ---- Past 32 bits -----------------------------------------------------------------

@pytest.mark.parametrize("t", [7, 90])
def test_a_head_past_two_to_the_31_bytes(t):
    """1.1 million rows of 2 048 codes: the last vocabulary rows, by streams and by
    tiles."""
    h, v = 2048, 1100000
    g = torch.Generator(device=DEV).manual_seed(t)
    w = torch.empty(v, h, dtype=torch.int8, device=DEV)
    w.random_(-127, 128, generator=g)
    ws = torch.rand(v, generator=g, device=DEV) * 1e-3
    x = torch.empty(t, h, dtype=torch.int8, device=DEV)
    x.random_(-127, 128, generator=g)
    xs = torch.rand(t, generator=g, device=DEV) * 1e-3
    z = lp.logits_int8(x, xs, w, ws, dtype=torch.float32)
    for a in (0, 1048560, v - 300):
        want = int8_head.logits_f32(x.cpu(), xs.cpu(), w[a:a + 300].cpu(), ws[a:a + 300].cpu())
        assert np.array_equal(z[:, a:a + 300].cpu().numpy(), want)
    ids = torch.full((t,), v - 1, device=DEV)
    got = lp.score_int8(x, xs, w, ws, ids)
    want = torch.log_softmax(z.double(), dim=1)[:, -1]
    assert (got.double() - want).abs().max() <= 2e-5 * (1 + want.abs().max())


def test_logits_past_two_to_the_32_bytes():
    """20 000 rows of 120 001 bf16 logits: 4.8 GB, the last rows and columns."""
    t, h, v = 20000, 64, 120001
    g = torch.Generator(device=DEV).manual_seed(1)
    w = torch.empty(v, h, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    ws = torch.rand(v, generator=g, device=DEV) * 1e-2
    x = torch.empty(t, h, dtype=torch.int8, device=DEV).random_(-127, 128, generator=g)
    xs = torch.rand(t, generator=g, device=DEV) * 1e-2
    z = lp.logits_int8(x, xs, w, ws)
    for r, c in ((0, 0), (17800, 60000), (t - 40, v - 200)):
        want = int8_head.logits_f32(x[r:r + 40].cpu(), xs[r:r + 40].cpu(), w[c:c + 200].cpu(),
                                    ws[c:c + 200].cpu())
        assert torch.equal(z[r:r + 40, c:c + 200].cpu().view(torch.int16),
                           torch.from_numpy(want).bfloat16().view(torch.int16))


def test_quantise_past_two_to_the_32_bytes():
    x = torch.empty(600000, 4097, dtype=torch.bfloat16, device=DEV)[:, :4096]
    x.zero_()
    x[-3:] = torch.randn(3, 4096, device=DEV).bfloat16()
    q, s = lp.quantize_int8(x)
    rq, rs = int8_head.quantize(x[-4:].float().cpu())
    assert np.array_equal(q[-4:].cpu().numpy(), rq) and np.array_equal(s[-4:].cpu().numpy(), rs)
    assert (s[:-3] == 0).all()


@pytest.mark.parametrize("how", [dict(), dict(top_p=0.9), dict(top_k=9), dict(min_p=0.05)], ids=str)
def test_verified_rows_past_32_bits(how):
    """Rows 2^28 elements apart, and the largest vocabulary."""
    b, d, v, ld = 4, 2, 5000, 1 << 28
    z = torch.empty(b * (d + 1) * ld, dtype=torch.bfloat16, device=DEV).as_strided(
        (b * (d + 1), v), (ld, 1))
    y = torch.empty(b * d * ld, dtype=torch.bfloat16, device=DEV).as_strided((b * d, v), (ld, 1))
    g = torch.Generator(device=DEV).manual_seed(4)
    z.copy_(3 * torch.randn(z.shape, generator=g, device=DEV))
    y.copy_(3 * torch.randn(y.shape, generator=g, device=DEV))
    ids = torch.randint(0, v, (b, d), generator=g, device=DEV)
    u = torch.rand(b, d + 1, generator=g, device=DEV)
    got = lp.verify(z, ids, u, y, **how)
    want = oracle_verify.verify(z.double().cpu().numpy(), ids.cpu().numpy(), u.cpu().numpy(),
                                y.double().cpu().numpy(), **how)
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    del z, y
    v = 1 << 20
    for dtype in (torch.float32, torch.float16):
        z = torch.randn(6, v, generator=g, device=DEV).to(dtype)
        y = (z.view(2, 3, v)[:, :2].reshape(4, v).float()
             + 0.3 * torch.randn(4, v, generator=g, device=DEV)).to(dtype)
        ids = y.argmax(dim=1).view(2, 2)
        u = torch.tensor([[0.99, 0.9, 0.999], [0.2, 0.99, 0.5]], device=DEV)
        got = lp.verify(z, ids, u, y, **how)
        want = oracle_verify.verify(z.double().cpu().numpy(), ids.cpu().numpy(), u.cpu().numpy(),
                                    y.double().cpu().numpy(), **how)
        assert np.array_equal(got[0].cpu().numpy(), want[0])


# ---- The most rows -----------------------------------------------------------------

def test_the_most_rows_quantised():
    x = torch.arange(16777215, device=DEV, dtype=torch.float32)[:, None] - 8e6
    q, s = lp.quantize_int8(x)
    assert torch.equal(s, x[:, 0].abs() * np.float32(np.float32(1) / np.float32(127)))
    # (|x| / scale is within a rounding of 127.)
    assert torch.equal(q[:, 0].long(), 127 * torch.sign(x[:, 0]).long())
    with pytest.raises(lp.LpError):
        lp.quantize_int8(torch.empty(16777216, 1, device=DEV))


def test_hundreds_of_thousands_of_tokens():
    t, v, h = 300001, 130, 40
    g = torch.Generator(device=DEV).manual_seed(2)
    w, ws = lp.quantize_int8(torch.randn(v, h, generator=g, device=DEV))
    x, xs = lp.quantize_int8(torch.randn(t, h, generator=g, device=DEV))
    z = lp.logits_int8(x, xs, w, ws, torch.float32)
    want = (x.float() @ w.float().t()) * xs[:, None] * ws  # (sums below 2^24: exact)
    assert torch.equal(z, want)
    ids = torch.arange(t, device=DEV) % v
    got = lp.score_int8(x, xs, w, ws, ids, check=True)
    exact = torch.log_softmax(z.double(), dim=1).gather(1, ids[:, None])[:, 0]
    assert (got.double() - exact).abs().max() <= 2e-5


@pytest.mark.parametrize("how", [dict(), dict(temperature=0.0), dict(top_p=0.6)], ids=str)
def test_the_most_sequences(how):
    """Without drafts each draws one token: as sample() would, but in index order."""
    b, v = 4194303, 3
    g = torch.Generator(device=DEV).manual_seed(2)
    z = torch.randn(b, v, generator=g, device=DEV)
    u = torch.rand(b, 1, generator=g, device=DEV)
    ids = torch.empty(b, 0, dtype=torch.int64, device=DEV)
    tokens, accepted, raw, proc = lp.verify(z, ids, u, check=True, **how)
    assert (accepted == 0).all()
    p = torch.softmax(z.double(), dim=1)
    if "top_p" in how:
        top, order = p.sort(dim=1, descending=True)
        gone = top.cumsum(dim=1) - top >= np.float64(np.float32(0.6))
        p = p.masked_fill(torch.zeros_like(gone).scatter(1, order, gone), 0.0)
    elif how:
        p = torch.zeros_like(p).scatter(1, z.argmax(dim=1, keepdim=True), 1.0)
    c = p.cumsum(dim=1)
    want = (c <= u.double() * c[:, -1:]).sum(dim=1)
    # (Borders within fp64's roundings of either side may fall to the other.)
    assert (tokens[:, 0] != want).sum() <= 2
    with pytest.raises((lp.LpError, ValueError)):
        lp.verify(torch.empty(b + 1, 1, device=DEV), torch.empty(b + 1, 0, dtype=torch.int64, device=DEV),
                  torch.empty(b + 1, 1, device=DEV))
