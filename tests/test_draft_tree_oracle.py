"""The draft-tree oracle against the framework's older definitions and against hand-made cases."""

import numpy as np

from oracle import draft_tree as D
from oracle import mla_oracle as O
from tests import tree_cases as T


def test_chain_is_token_causal_attention():
    """A chain of nodes behind a context is mla_attend's mask with one-token frames."""
    wl = T.workload(T.MAIN, 1, 40).scaled(n_heads=2)
    rng = np.random.default_rng(0)
    n, rows, first = 5, 20, 33                       # wraps the ring
    q = rng.standard_normal((1, n, 2, 576))
    cache = rng.standard_normal((1, 40, 576))
    win = np.array([[first, rows, n]])
    o, lse, _ = D.attend_tree(q, cache, win, None, 0.07, 512)
    g0 = first + 40                                  # token whose slot is `first`
    want_o, want_lse = O.attend_latent(q, cache, g0 + rows, g0, rows + n, 0.07, wl)[:2]
    np.testing.assert_allclose(o, want_o, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse, want_lse, rtol=1e-12)
    tri = np.tril(np.ones((1, n, n), dtype=bool))
    o2, _, _ = D.attend_tree(q, cache, win, tri, 0.07, 512)
    np.testing.assert_array_equal(o, o2)


def test_weights_of_a_row_sum_to_its_queries():
    rng = np.random.default_rng(1)
    q = rng.standard_normal((2, 3, 4, 80))
    cache = rng.standard_normal((2, 30, 80))
    win = np.array([[25, 9, 3], [4, 0, 2]])
    _, see = T.random_tree(rng, 2, 3)
    _, lse, _ = D.attend_tree(q, cache, win, see, 0.1, 64)
    w = D.attend_weight(q, cache, win, see, 0.1, lse, None, None, np.zeros((2, 30)))
    # every (node, head) hands out a total of one
    np.testing.assert_allclose(w.sum(1), [3 * 4, 2 * 4], rtol=1e-12)
    old = rng.random((2, 30))
    w2 = D.attend_weight(q, cache, win, see, 0.1, lse, None, old, old)
    at = D.slots(25, 9, 30)
    np.testing.assert_allclose(w2[0, at], old[0, at] + w[0, at], rtol=1e-12)
    tail = [(25 + 9 + i) % 30 for i in range(3)]
    np.testing.assert_array_equal(w2[0, tail], w[0, tail])


def test_evict_by_hand():
    S = 8
    cache = np.arange(S, dtype=float).reshape(1, S, 1) * np.ones((1, 1, 2))
    weight = np.array([[5.0, 1.0, np.nan, 4.0, 1.0, 0.5, 9.0, 9.0]])
    pos = np.array([[0, 1, 2, 3, 4, 5, 70, 71]])
    win = np.array([[0, 6, 2]])
    # position 5 is the newest: recent keeps row 5; sink keeps row 0; then 3 (4.0), 1 (1.0, lower row)
    c, w, wt, p = D.cache_evict(cache, win, weight, pos, 4, 1, 1)
    assert w.tolist() == [[0, 4, 0]]
    assert c[0, :4, 0].tolist() == [0, 1, 5, 3] and p[0, :4].tolist() == [0, 1, 5, 3]
    assert c[0, 4:, 0].tolist() == [4, 5, 6, 7]           # what lies past the end stays
    c, w, _, _ = D.cache_evict(cache, win, weight, pos, 6, 1, 1)
    assert w.tolist() == [[0, 6, 0]] and (c == cache).all()
    assert D.cache_evict(cache, win, weight, pos, 0, 1, 1)[1].tolist() == [[0, 0, 0]]


def test_accept_by_hand():
    S = 6
    cache = np.arange(S, dtype=float).reshape(1, S, 1)
    win = np.array([[4, 1, 4]])                            # context slot 4; nodes 5, 0, 1, 2
    acc = np.array([[False, True, False, True]])
    c, w, _, p = D.tree_accept(cache, win, None, np.arange(S)[None], acc)
    assert w.tolist() == [[4, 3, 0]]
    assert c[0, :, 0].tolist() == [0, 1, 2, 3, 4, 2] and p[0].tolist() == [0, 1, 2, 3, 4, 2]


def test_windows_are_clipped():
    assert D.clip_window((-3, 5, 2), 10, 4) == (0, 5, 2)
    assert D.clip_window((12, 99, 2), 10, 4) == (9, 10, 0)
    assert D.clip_window((3, 8, 7), 10, 4) == (3, 8, 2)
    assert D.clip_window((3, -1, -7), 10, 4) == (3, 0, 0)
