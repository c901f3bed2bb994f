"""The oracle of the operators around the paged cache against worked cases (CPU only)."""

import numpy as np

from oracle import cache_ops, paged


def test_rotation_of_one_pair_by_hand():
    x = np.zeros((1, 1, 4))
    x[0, 0] = [3, 5, 4, 7]                       # pairs (3, 4) and (5, 7)
    y = cache_ops.rotate(x, [[1], [2]], [0, 1], [np.pi / 2, np.pi / 2])
    assert np.allclose(y[0, 0], [-4, -5, 3, -7])


def test_rotation_keeps_scores_by_distance():
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((2, 1, 1, 16))
    axis, freq = [0, 1] * 4, [10.0 ** (-j / 4) for j in range(8)]

    def score(a, b):
        return np.sum(cache_ops.rotate(q[None], [[a[0]], [a[1]]], axis, freq) * cache_ops.rotate(k[None], [[b[0]], [b[1]]], axis, freq))

    assert np.isclose(score((5, 9), (2, 4)), score((105, 29), (102, 24)))
    assert not np.isclose(score((5, 9), (2, 4)), score((5, 9), (2, 5)))


def test_ancestors_by_hand():
    see = cache_ops.ancestors([-1, 0, 0, 1, -1, 4])
    want = np.array([[1, 0, 0, 0, 0, 0], [1, 1, 0, 0, 0, 0], [1, 0, 1, 0, 0, 0], [1, 1, 0, 1, 0, 0], [0, 0, 0, 0, 1, 0],
                     [0, 0, 0, 0, 1, 1]], bool)
    assert np.array_equal(see, want)
    v = cache_ops.tree_visible(see, 8)
    assert v[:, :2].all() and np.array_equal(v[:, 2:], want)
    assert np.array_equal(cache_ops.tree_visible(see, 4), want[:, 2:])      # more tokens than cached positions


def test_a_chain_is_causal_order():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((5, 2, 8)), rng.standard_normal((9, 1, 8)), rng.standard_normal((9, 1, 8))
    see = cache_ops.tree_visible(cache_ops.ancestors([-1, 0, 1, 2, 3]), 9)
    a = paged.attention(q, k, v, range(4, 9), 0.3, right=0)
    b = paged.attention(q, k, v, None, 0.3, see=see)
    assert all(np.array_equal(x, y) for x, y in zip(a, b))


def test_mass_sums_to_the_rows():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((6, 4, 8)), rng.standard_normal((10, 2, 8))
    pos = np.arange(4, 10)
    _, lse, _, _ = paged.attention(q, k, k, pos, 0.5, right=0)
    m, off = cache_ops.mass(q, lse, k, pos, 0.5, right=0)
    assert np.allclose(m.sum(axis=0), 12) and (off > 0).all() and off.max() < 1e-4      # two heads, six rows each
    lse[0] = -np.inf
    assert np.allclose(cache_ops.mass(q, lse, k, pos, 0.5, right=0)[0].sum(axis=0), 10)


def test_what_stays_by_hand():
    w = [0.0, 5.0, 1.0, 5.0, np.nan, 2.0, 0.0, 9.0]
    assert cache_ops.keep(w, 8, 0, 0) == list(range(8))
    assert cache_ops.keep(w, 3, 0, 0) == [1, 4, 7]
    assert cache_ops.keep(w, 4, 0, 0) == [1, 3, 4, 7]
    assert cache_ops.keep(w, 4, 1, 1) == [0, 1, 4, 7]
    assert cache_ops.keep(w, 4, 2, 2) == [0, 1, 6, 7]
    assert cache_ops.keep([1.0] * 5, 3, 0, 0) == [0, 1, 2]
