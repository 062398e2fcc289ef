"""lp_sample against the fp64 oracle. Tokens and kept counts are equal. The
scores are rounded to fp32 once: half a step relative (2^-24). The processed
score's mass is a sum of fp64 weights, or of weights in units of 2^-43 and
2^-44 a term: 1e-12 absolute inside the logarithm covers both. The raw score's
sum over the vocabulary has fp32 exponentials where a row goes by a short
list: 2^(z c - b) with c = log2 e / tau rounded to fp32 (half a step of the
temperature: 2^-24 of a difference of scores, at most |score| + ln V <= |score|
+ 12) and one rounding of the exponent x, ln2 * 2^-24 |x| of a weight; b is at
most 32 below the largest exponent and, weighted by the weights, the rest
averages at most log2 V <= 17.3: 35 * 2^-24; 2^-23 for the exponential; 31 + 6
additions of 2^-24 in a thread and across a wave. In all 86 * 2^-24 absolute
and 2^-24 of the score."""

import numpy as np
import pytest
import torch

import rollout_logprob_consistency_amd as lp
from oracle import logit_rows as ol

from .gpu_helpers import DEV
from .logits_helpers import dev, place, rows

pytestmark = pytest.mark.gpu
F32, I32 = torch.float32, torch.int32


def check(t, z, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, v_true=None):
    """Draws with the settings as tensors (arrays) or scalars, as given."""
    def arg(v, dtype):
        return dev(v, dtype) if isinstance(v, np.ndarray) else v
    got = lp.sample(t, dev(u, F32), arg(temperature, F32), arg(top_k, I32), arg(top_p, F32),
                    arg(min_p, F32), v_true=v_true)
    torch.cuda.synchronize()
    tok, raw, proc, kept = (g.cpu().numpy() for g in got)
    ref = ol.sample(z, np.asarray(u, np.float32), temperature, top_k, top_p, min_p)
    print("rows", z.shape, "kept", ref[3][:8])
    assert np.array_equal(kept, ref[3]), (kept, ref[3])
    assert np.array_equal(tok, ref[0]), (tok, ref[0])
    for g, r, log_err in ((raw, ref[1], 86 * 2.0 ** -24), (proc, ref[2], 1e-12)):
        assert np.array_equal(np.isnan(g), np.isnan(r))
        ok = ~np.isnan(r)
        assert np.all(np.abs(g[ok] - r[ok]) <= 2.0 ** -23 * np.abs(r[ok]) + log_err), (g, r)
    return got


def settings(rng, n):
    return dict(temperature=rng.choice(np.float32([0.0, 0.6, 1.0, 1.7]), n),
                top_k=rng.choice(np.int32([0, -1, 1, 2, 20, 300, 5000]), n),
                top_p=rng.choice(np.float32([1.0, 0.3, 0.9, 0.99, 0.0]), n),
                min_p=rng.choice(np.float32([0.0, 0.02, 0.3, 1e-30]), n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,v,pad,lead", [(1, 1, 0, 0), (3, 2, 1, 1), (5, 7, 0, 3), (9, 255, 2, 0),
                                          (9, 256, 0, 0), (4, 257, 0, 5), (33, 1000, 13, 0),
                                          (40, 4099, 0, 1), (12, 32003, 61, 2)])
def test_mixed_settings(dtype, n, v, pad, lead):
    t, z = rows(11 * v + n, n, v, dtype, pad=pad, lead=lead)
    rng = np.random.default_rng(v)
    check(t, z, rng.random(n, np.float32), **settings(rng, n))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("how", [dict(), dict(top_p=0.95), dict(temperature=0.7, top_k=20, top_p=0.8),
                                 dict(min_p=0.05), dict(temperature=0.0), dict(top_k=900),
                                 dict(temperature=2.5, top_k=3000, top_p=0.9)])
def test_a_language_models_vocabulary(dtype, how):
    t, z = rows(5, 4, 151936, dtype)
    check(t, z, [0.0, 0.37, 0.9, 1.0 - 2.0 ** -24], **how)


@pytest.mark.parametrize("masked", [0.3, 0.999])
def test_masked_tokens(masked):
    t, z = rows(7, 16, 5000, "fp32", masked=masked)
    z[3, :] = -np.inf
    z[3, 4321] = -7.0          # one token left
    z[4, :] = -np.inf          # none left
    t, z = place(z, "fp32")
    rng = np.random.default_rng(2)
    check(t, z, rng.random(16, np.float32), **settings(rng, 16))
    check(t, z, rng.random(16, np.float32), top_p=0.5)


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("kind", ["equal", "two_values", "narrow", "steps", "zeros"])
def test_crowded_buckets(dtype, kind):
    """More tokens within 1/32 nat than a list holds: whole vocabularies of
    equal values (ties by index), of two, and of distinct values."""
    rng = np.random.default_rng(4)
    n, v = 6, 20011
    z = {"equal": np.full((n, v), 1.5), "two_values": rng.choice([0.5, 0.5078125], (n, v)),
         "narrow": rng.normal(size=(n, v)) * 1e-3, "steps": np.floor(rng.normal(size=(n, v)) * 4) / 4,
         "zeros": rng.choice([0.0, -0.0], (n, v))}[kind]
    t, z = place(z, dtype)
    u = np.float32([0.0, 0.2, 0.5, 0.75, 0.9, 0.99999])
    check(t, z, u)
    check(t, z, u, top_p=0.5)
    check(t, z, u, top_k=9000, top_p=0.7)
    check(t, z, u, top_k=4097, min_p=0.99)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_borders_at_zero(dtype):
    """Logits on a grid of 1/32 around zero: every bucket's border is passed,
    the one between the zeros and the largest negative value among them."""
    rng = np.random.default_rng(6)
    n, v = 24, 700
    z = rng.integers(-3, 2, (n, v)) / 32.0
    z[rng.random((n, v)) < 0.1] *= -0.0
    t, z = place(z, dtype)
    u = ((np.arange(n) + 0.5) / n).astype(np.float32)
    check(t, z, u)
    check(t, z, u, top_k=600, top_p=0.8)
    for top_p in (0.2, 0.45, 0.7, 0.95):
        check(t, z, u, top_p=top_p)


def test_wide_rows():
    """Logits far below the maximum weigh nothing but count as kept; the
    largest finite logits; temperatures that push everything apart or together."""
    rng = np.random.default_rng(9)
    z = rng.normal(size=(6, 3001)) * 200
    z[1, 5] = 3.0e38
    z[2, :4] = [3.4e38, -3.4e38, 3.4e38, 0.0]
    t, z = place(z, "fp32")
    u = rng.random(6, np.float32)
    check(t, z, u)
    check(t, z, u, top_k=100)
    check(t, z, u, top_p=0.9, temperature=50.0)
    check(t, z, u, temperature=1e-3)
    check(t, z, u, temperature=1e30)
    check(t, z, u, min_p=1e-35)
    check(t, z, u, min_p=1.0)
    check(t, z, u, min_p=7.0)


@pytest.mark.parametrize("how", [dict(), dict(top_k=50), dict(top_p=0.8), dict(min_p=0.1)])
def test_the_smallest_temperature(how):
    """Logits of its own size, and logits beside which it is as good as zero."""
    tau = 2.0 ** -126
    rng = np.random.default_rng(12)
    z = rng.normal(size=(6, 9001)) * 4 * tau
    z[4:] = rng.normal(size=(2, 9001)) * 1e20
    t, z = place(z, "fp32")
    check(t, z, rng.random(6, np.float32), tau, **how)


def test_temperatures_that_are_none():
    t, z = rows(8, 5, 500)
    u = np.full(5, 0.5, np.float32)
    tau = np.float32([1.0, 1e-45, 2.0 ** -127, np.inf, 2.0 ** -126])
    for how in (dict(), dict(top_k=20), dict(min_p=0.05)):
        got = check(t, z, u, tau, **how)
        assert got[0].cpu().numpy()[1:4].tolist() == [-1, -1, -1]


def test_rows_without_a_draw():
    z = np.random.default_rng(1).normal(size=(8, 300))
    z[0, 7], z[1, 299], z[2, :], z[3, 0] = np.nan, np.inf, -np.inf, -np.inf
    t, zz = place(z, "fp32")
    u = np.float32([.5, .5, .5, .5, np.nan, .5, .5, .5])
    how = dict(temperature=np.float32([1, 1, 1, 1, 1, -1, np.nan, 1]),
               top_p=np.float32([1, 1, 1, 1, 1, 1, 1, np.nan]))
    check(t, zz, u, **how)
    bad = torch.zeros(1, dtype=I32, device=DEV)
    lp.sample(t, dev(u, F32), dev(how["temperature"], F32), top_p=dev(how["top_p"], F32),
              bad_rows=bad)
    assert bad.item() == 7
    with pytest.raises(ValueError, match="3 row"):
        lp.sample(t, torch.full((8,), 0.5, device=DEV), check=True)


def test_v_true_hides_the_padding():
    t, z = rows(3, 5, 1000, "bf16")
    z = z[:, :901]
    t[:, 901:] = 50.0
    check(t, z, [0.1, 0.3, 0.5, 0.7, 0.9], top_p=0.9, v_true=901)


def test_batch_invariance_and_alignment():
    """The same row drawn alone, in any place and at any alignment: the same bits."""
    for dtype in ("fp32", "bf16"):
        t, z = rows(21, 64, 10007, dtype)
        u = dev(np.random.default_rng(0).random(64), F32)
        ref = lp.sample(t, u, 0.8, 50, 0.95)
        for lead, pad in ((1, 0), (3, 5)):
            t2, _ = place(z, dtype, pad, lead)
            got = lp.sample(t2, u, 0.8, 50, 0.95)
            assert all(torch.equal(a, b) for a, b in zip(ref, got))
        for i in (0, 17, 63):
            got = lp.sample(t[i:i + 1], u[i:i + 1], 0.8, 50, 0.95)
            assert all(torch.equal(a[i:i + 1], b) for a, b in zip(ref, got))


def test_empty_and_wrong_arguments():
    z = torch.zeros(0, 10, device=DEV)
    assert lp.sample(z, torch.zeros(0, device=DEV))[0].shape == (0,)
    z, u = torch.zeros(4, 10, device=DEV), torch.zeros(4, device=DEV)
    for bad in (lambda: lp.sample(z.t(), u), lambda: lp.sample(z, u[:3]),
                lambda: lp.sample(z, u.double()), lambda: lp.sample(z[0].expand(4, 10), u),
                lambda: lp.sample(z.double(), u), lambda: lp.sample(z, u, v_true=11),
                lambda: lp.sample(z, u, v_true=0), lambda: lp.sample(z, u.cpu()),
                lambda: lp.sample(z, u, torch.ones(4, device=DEV, dtype=torch.float64))):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(temperature=-1.0), dict(top_p=float("nan"))):
        with pytest.raises(lp.LpError):
            lp.sample(z, u, **kw)
