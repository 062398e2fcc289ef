"""Pins of the 8-bit head's oracle: closed forms and brute force (CPU only)."""

from fractions import Fraction

import numpy as np
import pytest

from oracle import int8_head as o


def test_codes_of_a_known_row():
    q, s = o.quantize([[127.0, -127.0, 0.5, 1.5, 2.5, -0.5, 0.49, 63.2]])
    assert s[0] == 1.0
    assert q[0].tolist() == [127, -127, 0, 2, 2, 0, 0, 63]  # halves go to the even code


def test_rows_without_a_scale():
    q, s = o.quantize([[0.0, -0.0], [1.0, np.inf], [np.nan, 2.0], [2.0 ** -149, 0.0],
                       [64 * 2.0 ** -149, 2.0 ** -149]])
    assert s[0] == 0 and np.isnan(s[1]) and np.isnan(s[2]) and s[3] == 0
    assert s[4] == 2.0 ** -149 and q[4].tolist() == [64, 1]
    assert (q[:4] == 0).all()


@pytest.mark.parametrize("seed", range(3))
def test_codes_are_the_nearest_integers_of_real_quotients(seed):
    x = np.random.default_rng(seed).normal(size=(3, 50)).astype(np.float32)
    q, s = o.quantize(x)
    for r in range(3):
        for k in range(50):
            ratio = Fraction(float(x[r, k])) / Fraction(float(s[r]))
            best = min(range(-127, 128), key=lambda i: (abs(ratio - i), i % 2))
            assert q[r, k] == best


def test_logits_by_hand():
    x = np.array([[1, -2, 3]], np.int8)
    w = np.array([[4, 5, 6], [-128, 127, 0]], np.int8)
    assert o.sums(x, w).tolist() == [[12, -382]]
    z = o.logits(x, [0.5], w, [2.0, 0.25])
    assert z.tolist() == [[12.0, -47.75]]
    assert o.logits_f32(x, [0.5], w, [2.0, 0.25]).tolist() == z.tolist()


def test_scores_of_a_uniform_head():
    w = np.ones((8, 4), np.int8)
    z = o.logits(np.ones((2, 4), np.int8), [1.0, 3.0], w, np.ones(8))
    lp, lse = o.log_softmax_at(z, [0, 9], 2.0)
    assert lp[0] == pytest.approx(-np.log(8)) and np.isnan(lp[1])
    assert lse[1] == pytest.approx(12 / 2.0 + np.log(8))
