"""Pins of the oracle of drafted tokens' verification: worked cases and the
property it exists for (CPU only)."""

import numpy as np
import pytest

from oracle import verify as o

LOG = np.log([0.5, 0.3, 0.2])


def test_top_k_distribution_of_the_worked_token():
    p, raw = o.distribution(LOG, top_k=2)
    assert p == pytest.approx([0.625, 0.375, 0.0])
    assert raw == pytest.approx(LOG)


def test_a_greedy_row_is_one_token():
    p, raw = o.distribution([1.0, 3.0, 3.0], temperature=0.0)
    assert p.tolist() == [0, 1, 0]
    assert raw[1] == pytest.approx(-np.log(2 + np.exp(-2)))


def one(u, x, q=None, target=LOG):
    z = np.stack([target, LOG])
    return o.verify_sequence(z, [x], np.array(u), None if q is None else np.log([q]))


def test_accepted_and_rejected_by_hand():
    q = [0.2, 0.3, 0.5]
    # p(2) / q(2) = 0.4: accepted below it, and a token is drawn behind.
    assert one([0.39, 0.6], 2, q)[:2] == ([2, 1], 1)
    # Rejected above it: p - q is positive at token 0 alone.
    assert one([0.41, 0.99], 2, q)[:2] == ([0], 0)
    # A token that the target likes better than the draft is always accepted.
    assert one([0.999, 0.0], 0, q)[1] == 1
    # Without a draft model: p(x) itself, and the rest without x.
    assert one([0.29, 0.0], 1)[:2] == ([1, 0], 1)
    assert one([0.31, 0.72], 1)[:2] == ([2], 0)   # 0.5 of 0.7 lies below 0.72
    tokens, _, raw, proc = one([0.31, 0.70], 1)
    assert tokens == [0] and raw[0] == pytest.approx(np.log(0.5)) == pytest.approx(proc[0])


def test_nothing_beyond_the_draft():
    """p == q, and a drafted token that neither can give: from p itself."""
    p = [0.5, 0.5, 0.0]
    with np.errstate(divide="ignore"):
        z = np.log(p)
        got = o.verify_sequence(np.stack([z, z]), [2], np.array([0.0, 0.75]), z[None])
    assert got[:2] == ([1], 0)


def test_bad_sequences():
    z = np.stack([LOG, LOG])
    assert o.verify_sequence(z, [3], np.array([0.1, 0.1])) is None
    assert o.verify_sequence(z, [1], np.array([np.nan, 0.1])) is None
    assert o.verify_sequence(z, [1], np.array([0.1, 0.1]), z[:1] * np.nan) is None
    t, a, raw, _ = o.verify(np.tile(LOG, (4, 1)), np.array([[0], [1]]), np.full((2, 2), 0.1),
                            counts=[2, 0])
    assert a.tolist() == [-1, 0] and t[0].tolist() == [-1, -1] and np.isnan(raw[0]).all()
    assert t[1].tolist() == [0, -1] and raw[1, 1] == 0


@pytest.mark.parametrize("q", [[0.1, 0.2, 0.7], [0.5, 0.3, 0.2], [0.9, 0.05, 0.05], None])
def test_what_comes_out_is_distributed_as_the_target(q):
    """Over a fine grid of both random numbers, and drafted tokens weighed by q,
    the first token has the target's probabilities."""
    n = 200
    grid = (np.arange(n) + 0.5) / n
    weight = q if q is not None else [0.2, 0.5, 0.3]
    first = np.zeros(3)
    for x in range(3):
        for u in grid:
            accepted = one([u, 0.0], x, q)[1] == 1
            if accepted:
                first[x] += weight[x] / n
            else:
                for v in grid[::10]:
                    first[one([u, v], x, q)[0][0]] += weight[x] / n / 20
    assert first == pytest.approx([0.5, 0.3, 0.2], abs=0.03)
