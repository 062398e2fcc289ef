"""The operators on rows of logits at the ends of their documented ranges: the
largest vocabulary, more slices than a workgroup takes, vocabularies that end
inside a first or a last chunk."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import logit_rows as ol
from rollout_logprob_consistency_amd import _lib

from .gpu_helpers import DEV
from .logits_helpers import dev, place, rows
from .test_gpu_distill import DENSE_ERR, S_ERR

pytestmark = pytest.mark.gpu
F32 = torch.float32
MOST = _lib.SELECT_MAX_VOCAB


def check_draw(t, z, u, scores=True, **how):
    """Token and count are the oracle's; scores to its rounding as in test_gpu_sample.py."""
    got = lp.sample(t, dev(u, F32), **how)
    ref = ol.sample(z, np.asarray(u, np.float32), **how)
    print(z.shape, how, "kept", ref[3][:4], flush=True)
    assert np.array_equal(got[3].cpu().numpy(), ref[3])
    assert np.array_equal(got[0].cpu().numpy(), ref[0])
    if scores:
        for g, r, log_err in ((got[1], ref[1], 86 * 2.0 ** -24), (got[2], ref[2], 1e-12)):
            assert np.all(np.abs(g.cpu().numpy() - r) <= 2.0 ** -23 * np.abs(r) + log_err)
    return got


def check_top(t, z, k):
    got = lp.top_logprobs(t, k)
    ids, val, logp, _ = ol.top_logprobs(z, k)
    assert np.array_equal(got[0].cpu().numpy(), ids)
    assert np.array_equal(got[1].cpu().numpy(), val.astype(np.float32))
    assert np.all(np.abs(got[2].cpu().numpy() - logp) <= 2.0 ** -23 * np.abs(logp) + 86 * 2.0 ** -24)
    return got


HOW = (dict(), dict(top_p=0.9), dict(top_k=20, top_p=0.8), dict(temperature=0.0),
       dict(top_k=900), dict(min_p=0.05))


def largest(dtype):
    """Equal logits (a bucket's mass passes 2^63), a language model's, ties in steps."""
    rng = np.random.default_rng(3)
    z = np.stack([np.full(MOST, 1.5), rng.normal(size=MOST) * 2.2,
                  np.floor(rng.normal(size=MOST) * 4) / 4])
    z[1, rng.integers(0, MOST, 40)] += 12 * rng.random(40)
    return place(z, dtype)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_the_largest_vocabulary(dtype):
    t, z = largest(dtype)
    u = np.float32([0.25, 0.6, 0.999])
    for how in HOW:
        check_draw(t, z, u, **how)
    for k in (1, 64, 1024):
        check_top(t, z, k)


def test_the_largest_vocabulary_in_whole_rows():
    """260 rows (one workgroup each) of the same three: their bits."""
    t, _ = largest("fp32")
    n = 260
    many = t.repeat(n // 3 + 1, 1)[:n]
    u = dev(np.float32([0.25, 0.6, 0.999]), F32)
    us = u.repeat(n // 3 + 1)[:n]
    for how in HOW:
        few, got = lp.sample(t, u, **how), lp.sample(many, us, **how)
        for a, b in zip(few, got):
            assert torch.equal(a.repeat(n // 3 + 1)[:n], b), how
    for k in (64, 1024):
        few, got = lp.top_logprobs(t, k), lp.top_logprobs(many, k)
        for a, b in zip(few, got):
            assert torch.equal(a.repeat(n // 3 + 1, 1)[:n], b), k


@pytest.mark.parametrize("v", [30011, MOST])
def test_raw_scores_of_rows_by_buckets(v):
    """The raw score of rows that go by buckets: masses off by 1e-13 (2e-14 for
    the series, 2^-44 for the units, sums of 2 048 fp64 terms), one rounding to
    fp32, and nothing else but the tokens more than 39.9 nats below the
    maximum, which weigh 0."""
    rng = np.random.default_rng(8)
    z = rng.normal(size=(4, v)) * 2.2
    z[2] = -40.0                     # all of its rest is that far down
    z[2, 77] = 0.0
    z[3, 5] += 18.0
    t, z = place(z)
    u = np.float32([0.1, 0.5, 0.9, 0.3])
    far = np.array([np.exp(r - r.max())[r < r.max() - 39.9].sum() for r in z])
    assert far.max() <= MOST * np.exp(-39.9) < 5e-12
    for how in (dict(), dict(top_p=0.95), dict(top_k=900, top_p=0.9), dict(temperature=1.0, top_k=2000)):
        got, ref = lp.sample(t, dev(u, F32), **how), ol.sample(z, u, **how)
        assert np.array_equal(got[0].cpu().numpy(), ref[0])
        for g, r in ((got[1], ref[1]), (got[2], ref[2])):
            err = np.abs(g.double().cpu().numpy() - r)
            print(v, how, err)
            assert np.all(err <= 2.0 ** -24 * np.abs(r) + 1e-12 + far), (err, r)


@pytest.mark.parametrize("dtype,v", [("bf16", 2049), ("bf16", 3000), ("fp16", 3584), ("fp16", 4095),
                                     ("bf16", 4097), ("fp32", 1025), ("fp32", 2047),
                                     ("fp32", 8193), ("bf16", 16389)])
@pytest.mark.parametrize("n", [2, 300])
def test_vocabularies_that_end_inside_a_chunk(dtype, v, n):
    """A first chunk that some of a workgroup's waves have no token of, or a
    last chunk of a few: no wave's share is enough for a first bound on the
    list, which overflows where the row is longer than the list."""
    t, z = rows(v + n, n, v, dtype)
    rng = np.random.default_rng(n)
    u = rng.random(n, np.float32)
    for how in (dict(temperature=0.0), dict(top_k=1), dict(top_k=20), dict(top_k=157, top_p=0.9),
                dict(top_k=256), dict(top_k=257), dict(top_k=512, min_p=0.01), dict(min_p=0.02)):
        check_draw(t, z, u, **how)
    for k in (1, 157, 300, 1024):
        check_top(t, z, k)


@pytest.mark.parametrize("n", [1, 39])
def test_a_last_slice_of_a_short_chunk(n):
    t, z = rows(n, n, 200064, "bf16")
    u = np.random.default_rng(n).random(n, np.float32)
    for how in (dict(temperature=0.0), dict(top_k=20), dict(top_k=157)):
        check_draw(t, z, u, **how)
    check_top(t, z, 20)


def test_more_slices_than_a_workgroup_takes():
    """256 rows of 129 slices go by slices, as batches of 100 do; a row of 128
    goes by one workgroup where there are 256 of them."""
    for v in (128 * 4096, 128 * 4096 + 5):
        n, k = 256, 16
        g = torch.Generator(device=DEV).manual_seed(v)
        t = torch.randn(n, v, generator=g, device=DEV) * 2
        ids = torch.randint(0, v, (n, k), generator=g, device=DEV)
        ids[3, 4:9] = ids[3, 3]
        x = torch.randn(n, k, generator=g, device=DEV)
        w = torch.rand(n, generator=g, device=DEV)
        w[7] = 0
        loss, grad = lp.distill_step(t, ids, x, w)
        loss2, state = lp.distill_forward(t, ids, x)
        assert torch.equal(loss, loss2)
        assert torch.equal(lp.distill_backward(t, ids, x, state, w), grad)
        for a in range(0, n, 100):
            s = slice(a, a + 100)
            l3, g3 = lp.distill_step(t[s], ids[s], x[s], w[s])
            assert torch.equal(l3, loss[s]) and torch.equal(g3, grad[s])
        for r in (0, 3, 7, 255):
            logp = torch.log_softmax(t[r].double(), 0)
            q = torch.softmax(x[r].double(), 0)
            ref = (q * (q.log() - logp[ids[r]])).sum()
            assert (loss[r] - ref).abs() <= S_ERR + 2.0 ** -24 * ref.abs()
            want = torch.zeros(v, dtype=torch.float64, device=DEV)
            want.index_put_((ids[r],), q, accumulate=True)
            want = (logp.exp() - want) * w[r]
            tol = 2.0 ** -24 * want.abs() + DENSE_ERR * 1.01 * logp.exp() * w[r] + 2.0 ** -120
            assert ((grad[r].double() - want).abs() <= tol).all()
        assert not grad[7].any()


@pytest.mark.parametrize("n", [3, 300])
def test_both_sides_of_the_largest_short_list(n):
    t, z = rows(n, n, 30011, "bf16")
    u = np.random.default_rng(n).random(n, np.float32)
    for k in (400, 419, 420, 421, 512, 513):
        check_draw(t, z, u, top_k=k, top_p=0.97)
        got = lp.sample(t, dev(u, F32), 1.0, torch.full((n,), k, dtype=torch.int32, device=DEV), 0.97)
        assert all(torch.equal(a, b) for a, b in zip(got, lp.sample(t, dev(u, F32), top_k=k, top_p=0.97)))
    for k in (420, 421, 513):
        check_top(t, z, k)
