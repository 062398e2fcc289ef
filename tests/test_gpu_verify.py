"""Verification of drafted tokens on the GPU (lp_verify) against its fp64 oracle:
tokens and counts exactly, scores within their one rounding (and, for raw ones,
what the log-sum of a short list may be off by)."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import verify as oracle

from .gpu_helpers import DEV
from .logits_helpers import TYPES, dev, place, rows

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def batch(seed, b, d, v, dtype="fp32", model=True, noise=0.7, pad=0, lead=0, masked=0.0, **how):
    """A batch of drafted sequences: target rows, a draft that mostly agrees, its
    tokens drawn from its own distribution (with settings `how`)."""
    rng = np.random.default_rng(seed)
    z, exact = rows(seed, b * (d + 1), v, dtype, masked=masked, pad=pad, lead=lead)
    y = exact_y = None
    if model:
        near = exact.reshape(b, d + 1, v)[:, :d].reshape(b * d, v)
        y, exact_y = place(near + noise * rng.normal(size=near.shape), dtype, pad, lead)
    ids = np.zeros((b, d), np.int64)
    for i in range(b):
        one = {k: (x[i] if np.ndim(x) else x) for k, x in how.items()}
        for j in range(d):
            row = exact_y[i * d + j] if model else exact[i * (d + 1) + j]
            p = oracle.distribution(row, **one)[0]
            ids[i, j] = rng.choice(v, p=p / p.sum())
    u = rng.random((b, d + 1)).astype(np.float32)
    return z, y, ids, u, exact, exact_y


def check(z, y, ids, u, exact, exact_y, counts=None, **how):
    b, d = ids.shape
    on = {k: (dev(x, torch.int32 if k == "top_k" else torch.float32) if np.ndim(x) else x)
          for k, x in how.items()}
    got = lp.verify(z, dev(ids, torch.int64), dev(u, torch.float32), y,
                    None if counts is None else dev(counts, torch.int32), **on)
    want = oracle.verify(exact, ids, u, exact_y, counts, **how)
    compare(got, want)
    return got


def compare(got, want):
    tokens, accepted, raw, proc = (t.cpu().numpy() for t in got)
    assert np.array_equal(tokens, want[0]) and np.array_equal(accepted, want[1])
    assert np.array_equal(np.isnan(raw), np.isnan(want[2]))
    assert np.array_equal(np.isnan(proc), np.isnan(want[3]))
    # fp32's rounding; a short list's log-sum may be off by 210 * 2^-24.
    assert (np.nan_to_num(np.abs(raw - want[2])) <= E * np.abs(np.nan_to_num(want[2])) + 210 * E).all()
    assert (np.nan_to_num(np.abs(proc - want[3])) <= E * np.abs(np.nan_to_num(want[3])) + 1e-9).all()


SETTINGS = [dict(), dict(temperature=0.7), dict(temperature=1.4, top_p=0.9),
            dict(top_k=20, top_p=0.8), dict(top_k=1), dict(min_p=0.05), dict(temperature=0.0),
            dict(top_k=500), dict(top_k=200), dict(top_k=201, min_p=0.01),
            dict(top_k=600, top_p=0.95, min_p=0.01), dict(top_p=0.5, min_p=0.2),
            dict(top_p=0.0), dict(top_p=0.9, min_p=1.5), dict(temperature=0.2),
            dict(temperature=1e-3), dict(temperature=2.0 ** -126), dict(temperature=1e30),
            dict(temperature=1e-30, top_p=0.9), dict(temperature=1e4, min_p=0.5)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("how", SETTINGS, ids=str)
def test_settings(how, dtype):
    for model in (True, False):
        check(*batch(3, 5, 4, 5003, dtype, model, **how), **how)


@pytest.mark.parametrize("b,d,v", [(1, 0, 1), (1, 1, 1), (3, 2, 2), (4, 0, 300), (2, 63, 50),
                                   (7, 3, 4096), (6, 2, 4097), (2, 4, 20011), (70, 1, 1500),
                                   (1, 5, 151936)])
@pytest.mark.parametrize("how", [dict(), dict(top_p=0.9), dict(top_k=7)], ids=str)
def test_sizes(b, d, v, how):
    check(*batch(b + d, b, d, v, "bf16", True, **how), **how)
    check(*batch(b + d, b, d, v, "fp32", False, **how), **how)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad,lead", [(0, 1), (1, 0), (13, 5), (64, 0)])
def test_rows_of_any_stride(dtype, pad, lead):
    """What lies around the rows is NaN: reading it would show."""
    how = dict(top_p=0.9)
    check(*batch(1, 4, 3, 3001, dtype, True, pad=pad, lead=lead), )
    check(*batch(2, 4, 3, 3001, dtype, True, pad=pad, lead=lead, **how), **how)


@pytest.mark.parametrize("model", [True, False])
def test_ragged_sequences_with_settings_of_their_own(model):
    b, d, v = 40, 5, 4001
    rng = np.random.default_rng(9)
    how = dict(temperature=rng.choice(np.float32([0, 0.5, 1, 1.3]), b),
               top_k=rng.choice(np.int32([0, -1, 1, 30, 450, 5000]), b),
               top_p=rng.choice(np.float32([1, 0.3, 0.9, 0.99]), b),
               min_p=rng.choice(np.float32([0, 0, 0.02, 0.3]), b))
    data = batch(4, b, d, v, "bf16", model, **how)
    counts = rng.integers(0, d + 1, b).astype(np.int32)
    z, y, ids, u, exact, exact_y = data
    # What lies behind a sequence's drafts is not looked at.
    for i in range(b):
        z[i * (d + 1) + counts[i] + 1:(i + 1) * (d + 1)] = float("nan")
        if model:
            y[i * d + counts[i]:(i + 1) * d] = float("nan")
        ids[i, counts[i]:] = -5
        u[i, counts[i]:d] = np.nan
    got = check(z, y, ids, u, exact, exact_y, counts, **how)
    assert (got[1].cpu().numpy() >= 0).all()


@pytest.mark.parametrize("b,d,v", [(1366, 1, 70), (820, 2, 200), (5000, 0, 40), (1000, 3, 2500)])
def test_thousands_of_rows(b, d, v):
    """To both sides of 4 096, whole ones and others, some sequences without
    drafts, and one with a count that is none."""
    rng = np.random.default_rng(b)
    how = dict(temperature=rng.choice(np.float32([0, 0.7, 1]), b),
               top_k=rng.choice(np.int32([0, 0, 0, 9]), b),
               top_p=rng.choice(np.float32([1, 1, 0.9]), b),
               min_p=rng.choice(np.float32([0, 0, 0.1]), b))
    counts = rng.integers(0, d + 1, b).astype(np.int32)
    counts[17] = d + 1
    data = batch(b, b, d, v, "bf16", True, **how)
    got = check(*data, counts, **how)
    assert (got[1] < 0).nonzero().flatten().tolist() == [17]


@pytest.mark.parametrize("how", [dict(), dict(top_p=0.5), dict(top_k=300), dict(top_k=9001),
                                 dict(min_p=0.5), dict(min_p=1.0), dict(top_p=0.7, min_p=0.9),
                                 dict(temperature=0.0), dict(top_k=9001, top_p=0.6)], ids=str)
def test_rows_of_equal_logits(how):
    """Lists that overflow, buckets too full to list, ties by index."""
    b, d, v = 2, 2, 20011
    rng = np.random.default_rng(1)
    for levels in (1, 3, 40):
        z, exact = place(np.floor(rng.random((b * (d + 1), v)) * levels) / 16, "bf16")
        y, exact_y = place(np.floor(rng.random((b * d, v)) * levels) / 16, "bf16")
        ids = rng.integers(0, v, (b, d))
        u = rng.random((b, d + 1)).astype(np.float32)
        check(z, y, ids, u, exact, exact_y, **how)
        check(z, None, ids, u, exact, None, **how)


@pytest.mark.parametrize("how", [dict(), dict(top_p=0.95), dict(top_k=40), dict(min_p=0.01)], ids=str)
def test_masked_tokens(how):
    check(*batch(5, 6, 3, 3000, "fp16", True, masked=0.6, **how), **how)
    # One token left; and a drafted token that is masked in the target.
    z = np.full((4, 50), -np.inf)
    z[[0, 1, 2, 3], [7, 8, 9, 9]] = 1.0
    y = np.full((2, 50), -np.inf)
    y[[0, 1], [7, 3]] = 0.5
    zt, exact = place(z)
    yt, exact_y = place(y)
    got = check(zt, yt, np.array([[7], [3]]), np.full((2, 2), 0.5, np.float32), exact, exact_y,
                **how)
    assert got[0].tolist() == [[7, 8], [9, -1]] and got[1].tolist() == [1, 0]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("how", [dict(), dict(min_p=0.1), dict(temperature=0.5)], ids=str)
def test_rows_that_hold_no_number(dtype, how):
    """A NaN or an infinity in any place of a row that is summed whole, beside masked
    tokens: the sequence has no verdict, and its neighbours have theirs."""
    b, d, v = 9, 1, 9001
    z, y, ids, u, exact, exact_y = batch(3, b, d, v, dtype, True, masked=0.5, **how)
    for row, at, value in ((1, 0, np.nan), (4, v - 1, np.nan), (8, 4097, np.inf), (10, 77, -np.nan)):
        z[row, at] = value
        exact[row, at] = value
    y[5, 8000] = exact_y[5, 8000] = np.nan
    y[7] = exact_y[7] = -np.inf
    got = check(z, y, ids, u, exact, exact_y, **how)
    assert (got[1] < 0).nonzero().flatten().tolist() == [0, 2, 4, 5, 7]


LOWEST = {"fp32": np.finfo(np.float32).min, "bf16": -(2.0 - 2.0 ** -7) * 2.0 ** 127, "fp16": -65504.0}


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("how", [dict(), dict(temperature=0.3, top_p=0.9), dict(top_k=30),
                                 dict(min_p=0.1), dict(temperature=0.0)], ids=str)
def test_masks_of_the_lowest_value(dtype, how):
    """Masks that are finite: behind the language's tokens, in all but one place, and
    throughout; and rows at the type's other end."""
    b, d, v = 6, 3, 5003
    rng = np.random.default_rng(12)
    z = np.floor(8 * rng.normal(size=(b * (d + 1), v))) / 4
    low = LOWEST[dtype]
    z[:, ::3] = low
    z[5], z[6], z[7] = low, low, -low
    z[6, 4321] = 1.5
    z[8, 1:] = low
    z[9, 2500:] = -np.inf
    y = z.reshape(b, d + 1, v)[:, :d].reshape(b * d, v).copy()
    y[rng.random(y.shape) < 0.2] = 0.5
    y[4] = low
    zt, z = place(z, dtype)
    yt, y = place(y, dtype)
    ids = rng.integers(0, v, (b, d))
    for i in range(b):
        for j in range(d):
            p = oracle.distribution(y[i * d + j], **how)[0]
            ids[i, j] = rng.choice(v, p=p / p.sum())
    check(zt, yt, ids, rng.random((b, d + 1)).astype(np.float32), z, y, **how)


def test_the_same_rows_are_always_accepted():
    z, y, ids, u, exact, _ = batch(6, 5, 4, 2000, noise=0.0)
    got = lp.verify(z, dev(ids, torch.int64), dev(np.full_like(u, 1.0), torch.float32), y)
    assert (got[1] == 4).all()


def test_nothing_beyond_the_draft():
    """Equal rows and a drafted token that neither model gives."""
    z = np.zeros((2, 9000))
    z[:, 5] = -np.inf
    zt, exact = place(z)
    yt, exact_y = place(z[:1])
    for last in (0.0, 0.25, 0.99999, 1.0):
        check(zt, yt, np.array([[5]]), np.array([[0.0, last]], np.float32), exact, exact_y)


def test_what_comes_out_is_distributed_as_the_target():
    """Over a grid of 64 x 64 random numbers and every drafted token, weighed by
    the draft's probabilities, the first token has the target's: each step of
    the grid is off by at most one part in 64, and a token takes part in the
    acceptance and in the draw."""
    v, n = 5, 64
    z = np.array([1.0, 0.2, -0.5, 0.9, -2.0])
    y = np.array([0.1, 1.1, -0.3, 0.0, 0.4])
    p, q = (np.exp(x) / np.exp(x).sum() for x in (z, y))
    grid = ((np.arange(n) + 0.5) / n).astype(np.float32)
    u = np.stack(np.meshgrid(grid, grid, indexing="ij"), -1).reshape(-1, 2)
    for y_rows, weight in ((y, q), (None, np.array([0.1, 0.2, 0.3, 0.25, 0.15]))):
        first = np.zeros(v)
        b = u.shape[0]
        zt = dev(np.tile(z, (2 * b, 1)), torch.float32)
        yt = None if y_rows is None else dev(np.tile(y, (b, 1)), torch.float32)
        for x in range(v):
            got = lp.verify(zt, torch.full((b, 1), x, device=DEV), dev(u, torch.float32), yt)
            first += weight[x] * np.bincount(got[0][:, 0].cpu().numpy(), minlength=v) / b
        assert np.abs(first - p).max() <= 2.0 / n


def test_sequences_without_a_verdict():
    b, d, v = 12, 2, 500
    z, y, ids, u, exact, exact_y = batch(8, b, d, v)
    counts = np.full(b, d, np.int32)
    tau = np.ones(b, np.float32)
    top_p = np.ones(b, np.float32)
    counts[0], counts[1] = -1, d + 1
    ids[2, 0], ids[3, 1] = -1, v
    u[4, 1] = np.nan
    u[5, d] = np.nan
    z[6 * (d + 1) + 2, 9] = exact[6 * (d + 1) + 2, 9] = float("nan")
    z[7 * (d + 1), 0] = exact[7 * (d + 1), 0] = float("inf")
    y[8 * d + 1] = exact_y[8 * d + 1] = float("-inf")
    tau[9], top_p[10] = -1.0, np.nan
    bad = torch.full((1,), 3, dtype=torch.int32, device=DEV)
    how = dict(temperature=dev(tau, torch.float32), top_p=dev(top_p, torch.float32))
    args = (z, dev(ids, torch.int64), dev(u, torch.float32), y, dev(counts, torch.int32))
    got = lp.verify(*args, **how, bad_rows=bad)
    compare(got, oracle.verify(exact, ids, u, exact_y, counts, tau, 0, top_p, 0.0))
    assert got[1].tolist()[:11] == [-1] * 11 and got[1][11] >= 0 and bad.item() == 14
    with pytest.raises(ValueError, match="^11 row"):
        lp.verify(*args, **how, check=True)


@pytest.mark.parametrize("how", [dict(), dict(top_p=0.9), dict(top_k=30), dict(min_p=0.02)], ids=str)
def test_results_do_not_depend_on_the_batch(how):
    b, d, v = 150, 2, 9001
    z, y, ids, u, _, _ = batch(10, b, d, v, "bf16")
    ids, u = dev(ids, torch.int64), dev(u, torch.float32)
    whole = lp.verify(z, ids, u, y, **how)
    for lo, hi in ((0, 1), (3, 9), (20, 120), (149, 150)):
        part = lp.verify(z[lo * (d + 1):hi * (d + 1)], ids[lo:hi].contiguous(),
                         u[lo:hi].contiguous(), y[lo * d:hi * d], **how)
        for x, w in zip(part, whole):
            assert torch.equal(x, w[lo:hi])


def test_greedy_is_samples_greedy():
    z, y, ids, u, _, _ = batch(12, 20, 3, 3000, "bf16", temperature=0.0)
    got = lp.verify(z, dev(ids, torch.int64), dev(u, torch.float32), y, temperature=0.0)
    token, logprob, _, _ = lp.sample(z, torch.zeros(80, device=DEV), 0.0)
    there = got[0] >= 0
    assert torch.equal(got[0][there], token.view(20, 4)[there])
    assert torch.equal(got[2][there], logprob.view(20, 4)[there])
    assert (got[3] == 0).all()


def test_a_workspace_of_a_larger_batch_serves():
    from rollout_logprob_consistency_amd._lib import lib
    z, y, ids, u, exact, exact_y = batch(13, 3, 2, 5000)
    ws = torch.empty(lib().lp_verify_workspace_bytes(50, 6, 9000, 0), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)
    got = lp.verify(z, dev(ids, torch.int64), dev(u, torch.float32), y, workspace=ws)
    compare(got, oracle.verify(exact, ids, u, exact_y))


def test_no_sequences():
    got = lp.verify(torch.empty(0, 100, device=DEV), torch.empty(0, 3, dtype=torch.int64, device=DEV),
                    torch.empty(0, 4, device=DEV))
    assert [tuple(t.shape) for t in got] == [(0, 4), (0,), (0, 4), (0, 4)]


def test_refusals_on_the_device():
    z, y, ids, u, _, _ = batch(14, 2, 2, 300)
    ids, u = dev(ids, torch.int64), dev(u, torch.float32)
    for args, text in (((z[:5], ids, u, y), "rows"), ((z, ids, u[:, :2].contiguous(), y), "u must"),
                       ((z, ids.int(), u, y), "draft_ids"), ((z, ids, u, y[:3]), "draft_logits"),
                       ((z, ids, u, y.half()), "draft_logits"), ((z, ids, u, y[:, :299]), "draft_logits"),
                       ((z, ids, u, y, torch.zeros(2, device=DEV)), "counts")):
        with pytest.raises(ValueError, match=text):
            lp.verify(*args)
    with pytest.raises(ValueError, match="at most 63"):
        lp.verify(z, torch.zeros(2, 64, dtype=torch.int64, device=DEV), u)
    with pytest.raises(lp.LpError):
        lp.verify(z, ids, u, y, temperature=-1.0)
