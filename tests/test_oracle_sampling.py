"""Pins of the sampling oracle (oracle/sampling.py): closed forms, a hand-worked example, numpy's inverse CDF, the
interval of u that draws each token, and the greedy limits."""
import numpy as np
import pytest

from oracle.accept import accept
from oracle.sampling import accept_sampled, kept_ids, sample_row


def test_hand_worked_row():
    # weights at T = 1: ids 0..4 -> 1, 2, 8, 4, 1 (of 16); order: 2, 3, 1, 0, 4
    x = np.log([1.0, 2.0, 8.0, 4.0, 1.0])
    assert kept_ids(x, 1.0)[0].tolist() == [0, 1, 2, 3, 4]
    assert kept_ids(x, 1.0, top_k=3)[0].tolist() == [1, 2, 3]
    assert kept_ids(x, 1.0, top_k=4)[0].tolist() == [0, 1, 2, 3]       # of the equal ids 0 and 4 the lower one
    assert kept_ids(x, 1.0, top_p=0.74)[0].tolist() == [2, 3]           # 8 + 4 = 12 of 16
    assert kept_ids(x, 1.0, top_p=0.76)[0].tolist() == [1, 2, 3]
    assert kept_ids(x, 1.0, min_p=0.2)[0].tolist() == [1, 2, 3]         # at least 1.6
    assert kept_ids(x, 1.0, top_k=3, top_p=0.8)[0].tolist() == [2, 3]   # 12 of the 14 that top-k kept
    assert kept_ids(x, 1.0, top_p=0.0)[0].tolist() == [2]
    assert [sample_row(x, u, 1.0)[0] for u in (0.0, 0.05, 0.07, 0.2, 0.6, 0.7, 0.93, 0.94)] == [0, 0, 1, 2, 2, 3, 3, 4]
    tok, lp = sample_row(x, 0.9, 1.0, top_k=3)
    assert tok == 3 and np.isclose(lp, np.log(4 / 14))


def test_uniform_row_is_a_ruler():
    x = np.full(10, -3.0)
    assert [sample_row(x, k / 16, 0.7)[0] for k in range(16)] == [10 * k // 16 for k in range(16)]
    assert sample_row(x, 0.99, 0.7, top_k=4) == (3, np.log(0.25))


def test_geometric_row_closed_form():
    # w_v = 2^-v: the mass of the first n of 40 is (2 - 2^(1-n)) / (2 - 2^-39)
    x = -np.log(2.0) * np.arange(40)
    for n in (1, 3, 9):
        edge = (2 - 2.0 ** (1 - n)) / (2 - 2.0 ** -39)
        assert kept_ids(x, 1.0, top_p=edge * (1 - 1e-9))[0].size == n
        assert kept_ids(x, 1.0, top_p=edge * (1 + 1e-9))[0].size == n + 1


def test_every_token_owns_an_interval_of_u_as_wide_as_its_probability():
    rng = np.random.default_rng(0)
    x = rng.standard_normal(50) * 2
    ids, w = kept_ids(x, 0.8, top_k=20, top_p=0.9, min_p=0.01)
    p = w / w.sum()
    lo = np.concatenate([[0], np.cumsum(p)[:-1]])
    for i, a, q in zip(ids, lo, p):
        for u in (a + 1e-9, a + 0.5 * q, a + q - 1e-9):
            tok, lp = sample_row(x, u, 0.8, 20, 0.9, 0.01)
            assert tok == i and np.isclose(lp, np.log(q))


def test_without_filters_it_is_numpys_inverse_cdf():
    rng = np.random.default_rng(1)
    for _ in range(50):
        x, u, t = rng.standard_normal(30), rng.random(), rng.uniform(0.3, 2)
        p = np.exp(x / t) / np.exp(x / t).sum()
        assert sample_row(x, u, t)[0] == int(np.searchsorted(np.cumsum(p), u, side="right"))


def test_greedy_limits():
    x = np.array([1.0, 3.0, 3.0, 2.0])
    assert sample_row(x, 0.999, 0.0) == (1, 0.0)
    assert sample_row(x, 0.999, 1.0, top_k=1) == (1, 0.0)
    assert sample_row(x, 0.999, 1.0, min_p=1.0)[0] == 2  # both maxima survive
    assert sample_row(x, 0.5, 1e-30)[0] == 2


def test_masked_rows():
    inf = np.inf
    assert sample_row([-inf, -inf], 0.5, 1.0) == (-1, -inf)
    assert sample_row([np.nan, -inf], 0.5, 0.0) == (-1, -inf)
    assert sample_row([-inf, 2.0, np.nan], 0.99, 1.0) == (1, 0.0)
    assert [sample_row([0.0, inf, 1.0, inf], u, 1.0)[0] for u in (0.0, 0.49, 0.5, 0.99)] == [1, 1, 3, 3]


@pytest.mark.parametrize("seed", range(4))
def test_walk_with_temperature_zero_is_the_greedy_walk(seed):
    rng = np.random.default_rng(seed)
    B, N, V, D = 3, 12, 6, 5
    parent = np.array([[-1] + [int(rng.integers(0, i)) for i in range(1, N)] for _ in range(B)])
    token = rng.integers(0, V, (B, N))
    x = rng.standard_normal((B, N, V))
    acc, path, bonus = accept(token, parent, x, D)
    got = accept_sampled(token, parent, x, rng.random((B, D + 1)), D, np.zeros(B))
    assert np.array_equal(got[0], acc) and np.array_equal(got[1], path) and np.array_equal(got[2], bonus)
    assert not got[3].any()


def test_walk_follows_the_drawn_tokens():
    # root's children carry tokens 0 and 1; u decides which; the child's row then ends the walk
    token = np.array([[9, 0, 1, 0]])
    parent = np.array([[-1, 0, 0, 2]])
    x = np.log(np.array([[[1.0, 3.0], [1.0, 1.0], [1.0, 1e-9], [1.0, 1.0]]]))
    acc, path, bonus, lp = accept_sampled(token, parent, x, np.array([[0.2, 0.7, 0.1]]), 2, np.ones(1))
    assert acc[0] == 1 and path[0].tolist() == [0, 1, -1] and bonus[0] == 1
    assert np.allclose(lp[0], [np.log(0.25), np.log(0.5), 0])
    acc, path, bonus, lp = accept_sampled(token, parent, x, np.array([[0.3, 0.7, 0.1]]), 2, np.ones(1))
    assert acc[0] == 2 and path[0].tolist() == [0, 2, 3] and bonus[0] == 0
