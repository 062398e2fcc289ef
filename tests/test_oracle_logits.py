"""Pins of the fp64 oracle for the operators on rows of logits: closed forms,
printed values, brute force, and gradients by differences."""

import itertools

import numpy as np
import pytest

from oracle import logit_rows as ol


def test_top_k_example_of_the_page():
    # Probabilities (0.5, 0.3, 0.2); two kept: (0.625, 0.375, 0).
    z = np.log([0.5, 0.3, 0.2])
    tok, lp, proc, kept = ol.sample_row(z, 0.0, top_k=2)
    assert (tok, kept) == (0, 2)
    assert np.isclose(np.exp(lp), 0.5) and np.isclose(np.exp(proc), 0.625)
    tok, lp, proc, kept = ol.sample_row(z, 0.63, top_k=2)
    assert (tok, kept) == (1, 2)
    assert np.isclose(np.exp(lp), 0.3) and np.isclose(np.exp(proc), 0.375)


@pytest.mark.parametrize("top_k,top_p,min_p,kept", [
    (0, 1.0, 0.0, 4), (3, 1.0, 0.0, 3), (0, 0.5, 0.0, 1), (0, 0.51, 0.0, 2), (0, 0.75, 0.0, 2),
    (0, 0.0, 0.0, 1), (0, 1.0, 0.5, 2), (0, 1.0, 0.51, 1), (0, 1.0, 2.0, 1),
    # the nucleus is of what top-k left: 0.75 of (0.5, 0.25) / 0.75 is 0.5625
    (2, 0.75, 0.0, 2), (2, 0.66, 0.0, 1), (9, 1.0, 0.0, 4)])
def test_filters_on_halving_weights(top_k, top_p, min_p, kept):
    z = np.log([0.5, 0.25, 0.125, 0.125])
    assert ol.sample_row(z, 0.0, 1.0, top_k, top_p, min_p)[3] == kept


def test_draw_is_the_inverse_of_the_sorted_distribution():
    z = np.log([0.125, 0.5, 0.125, 0.25])       # order 1, 3, 0, 2
    for u, tok in ((0.0, 1), (0.49, 1), (0.5, 3), (0.74, 3), (0.75, 0), (0.874, 0), (0.875, 2),
                   (0.999, 2), (1.0, 2), (-3.0, 1)):
        assert ol.sample_row(z, u)[0] == tok, u
    counts = np.bincount([ol.sample_row(z, (i + 0.5) / 800)[0] for i in range(800)], minlength=4)
    assert counts.tolist() == [100, 400, 100, 200]


def test_ties_masks_and_rows_without_a_draw():
    assert ol.sample_row([1.0, 2.0, 2.0, -np.inf], 0.0)[0] == 1
    assert ol.sample_row([0.0, -0.0, 0.0], 0.5)[0] == 1
    assert ol.sample_row([1.0, 2.0, 2.0, -np.inf], 0.5)[3] == 3
    assert ol.sample_row([5.0, 7.0], 0.9, temperature=0.0)[::3] == (1, 1)
    for z in ([np.nan, 0.0], [np.inf, 0.0], [-np.inf, -np.inf]):
        assert ol.sample_row(z, 0.5)[0] == -1
    assert ol.sample_row([0.0, 1.0], 0.5, temperature=-1.0)[0] == -1
    assert ol.sample_row([0.0, 1.0], np.nan)[0] == -1


def test_top_logprobs_brute_force():
    z = np.array([[0.5, 2.0, 2.0, -np.inf, 1.0]])
    ids, val, lp, lse = ol.top_logprobs(z, 5, 2.0)
    assert ids.tolist() == [[1, 2, 4, 0, -1]]
    assert val[0].tolist() == [2.0, 2.0, 1.0, 0.5, -np.inf]
    assert np.isclose(lse[0], np.log(sum(np.exp(np.array([0.25, 1.0, 1.0, 0.5])))))
    assert np.isclose(np.exp(lp[0]).sum(), 1.0)


def test_top_logprobs_of_large_logits():
    """ln 3 is not lost beside logits whose fp64 neighbours are 2^-13 apart and more."""
    for z in (1e12, 2.0 ** 60, -1e15):
        lp = ol.top_logprobs(np.full((1, 3), z), 2)[2]
        assert np.all(np.abs(lp + np.log(3)) <= 1e-15), (z, lp)


def test_distill_of_a_full_list_is_the_divergence():
    rng = np.random.default_rng(0)
    z, t = rng.normal(size=6), rng.normal(size=6)
    p, q = np.exp(z) / np.exp(z).sum(), np.exp(t) / np.exp(t).sum()
    loss, grad = ol.distill_row(z, np.arange(6), t)
    assert np.isclose(loss, (q * np.log(q / p)).sum())
    assert np.allclose(grad, p - q)
    # One entry of weight 1: the negative logprob of a token.
    loss, _ = ol.distill_row(z, np.array([4]), np.array([0.0]), renormalize=False)
    assert np.isclose(loss, -np.log(p[4]))


def test_distill_entries_that_are_absent_repeated_or_outside():
    z = np.array([0.3, -1.0, 2.0])
    a = ol.distill_row(z, np.array([2, -1, 0]), np.array([1.0, np.nan, 0.5]))
    b = ol.distill_row(z, np.array([2, 0]), np.array([1.0, 0.5]))
    assert a[0] == b[0] and np.array_equal(a[1], b[1])
    half = np.log(0.5)
    a = ol.distill_row(z, np.array([1, 1]), np.array([half, half]), renormalize=False)
    b = ol.distill_row(z, np.array([1]), np.array([0.0]), renormalize=False)
    assert np.allclose(a[1], b[1])
    assert ol.distill_row(z, np.array([-1, -1]), np.zeros(2))[0] == 0.0
    assert np.isnan(ol.distill_row(z, np.array([3]), np.zeros(1))[0])
    assert np.isnan(ol.distill_row(z, np.array([-2]), np.zeros(1))[0])


@pytest.mark.parametrize("renormalize,tau", itertools.product([True, False], [1.0, 0.5, 2.0]))
def test_distill_gradient_by_differences(renormalize, tau):
    rng = np.random.default_rng(3)
    z = rng.normal(size=7)
    ids = np.array([3, 0, -1, 6, 3])
    t = rng.normal(size=5) - (0.0 if renormalize else 2.0)
    _, grad = ol.distill_row(z, ids, t, tau, renormalize)
    h = 1e-5  # central differences: h^2 |f'''| / 6 ~ 1e-10 / tau^3, rounding 1e-16 / h = 1e-11
    for v in range(7):
        d = np.zeros(7)
        d[v] = h
        up = ol.distill_row(z + d, ids, t, tau, renormalize)[0]
        dn = ol.distill_row(z - d, ids, t, tau, renormalize)[0]
        assert abs((up - dn) / (2 * h) - grad[v]) < 5e-9
