"""Pins of oracle/paged.py: against the cascade's oracle, brute-force loops, closed forms."""
import numpy as np
import pytest

import oracle
from oracle import paged


def test_slots_follow_the_block_table():
    np.testing.assert_array_equal(paged.slots([5, 0, 3], [0, 15, 16, 40, 47], 16),
                                  [80, 95, 0, 56, 63])


def test_decode_is_the_last_row_of_causal_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(9, 8, 16)), rng.normal(size=(9, 2, 16)), rng.normal(size=(9, 2, 16))
    none = np.zeros((0, 2, 16))
    ref, ref_lse = oracle.suffix_attention(q, none, none, k, v, 0.25)
    out, lse, w = paged.decode(q[-1], k, v, 0.25)
    np.testing.assert_allclose(out, ref[-1], rtol=1e-12)
    np.testing.assert_allclose(lse, ref_lse[-1], rtol=1e-12)
    np.testing.assert_allclose(w.sum(1), [4, 4], rtol=1e-12)


def test_scores_are_column_sums_of_the_softmax():
    rng = np.random.default_rng(1)
    n, hq, hkv, d = 7, 4, 2, 8
    q, k = rng.normal(size=(n, hq, d)), rng.normal(size=(n, hkv, d))
    z = np.einsum("ihd,jhd->hij", q, k[:, np.arange(hq) // 2])
    for causal in (False, True):
        m = np.where(np.tril(np.ones((n, n), bool)), z, -np.inf) if causal else z
        p = np.exp(m) / np.exp(m).sum(-1, keepdims=True)
        lse = np.log(np.exp(m).sum(-1)).T
        got = paged.scores(q, k, lse, 1.0, causal)
        np.testing.assert_allclose(got, p.reshape(hkv, 2, n, n).sum((1, 2)), rtol=1e-12)
        got = paged.scores(q, k, lse, 1.0, causal, window=3)
        np.testing.assert_allclose(got, p.reshape(hkv, 2, n, n)[:, :, -3:].sum((1, 2)), rtol=1e-12)


@pytest.mark.parametrize("budget,recent", [(1, 0), (1, 1), (4, 2), (6, 0), (9, 3), (20, 5)])
def test_evict_against_a_loop(budget, recent):
    x = np.array([3.0, np.nan, 1.0, 3.0, -np.inf, 0.5, 3.0, 2.0, 9.0])
    n = 9
    new = min(n, budget)
    last = min(recent, new)
    left, kept = list(range(n - last)), []
    for _ in range(new - last):
        best = left[0]
        for j in left:
            a, b = (-np.inf if np.isnan(x[i]) else x[i] for i in (j, best))
            if a > b:
                best = j
        left.remove(best)
        kept.append(best)
    np.testing.assert_array_equal(paged.evict(x, n, budget, recent),
                                  sorted(kept) + list(range(n - last, n)))


def test_append_round_trip():
    rng = np.random.default_rng(2)
    pages = np.zeros((4, 16, 2, 8))
    new = rng.normal(size=(5, 2, 8))
    got = paged.append(pages, new, [0, 3, 5], [15, 0], np.array([[2, 0], [3, 1]]))
    flat = got.reshape(-1, 2, 8)
    np.testing.assert_array_equal(flat[[47, 0, 1, 48, 49]], new)
    assert np.count_nonzero(flat.any((1, 2))) == 5
