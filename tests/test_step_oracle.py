"""The oracle of acceptance and pages, pinned: closed forms, hand-worked
cases and invariants (CPU)."""
import itertools

import numpy as np
import pytest

from oracle import step_oracle as so


def _softmax(z):
    w = np.exp(z - z.max())
    return w / w.sum()


def test_accepting_a_drawn_token_leaves_the_target_distribution():
    """One drafted token from g, uniform u and v: summing over the token and
    integrating over u and v on a fine grid gives p back (rejection rule)."""
    z = np.array([[0.3, -1.0, 1.2, 0.0], [0.0, 0.0, 0.0, 0.0]])
    p = _softmax(z[0])
    g = np.array([0.5, 0.1, 0.1, 0.3])
    grid = (np.arange(400) + 0.5) / 400
    got = np.zeros(4)
    for x in range(4):
        for u in grid:
            path, token, _ = so.accept_sequence(z, [g, g], [0, x], [-1, 0], [0, u], 0.5, 1.0)
            if len(path) == 2:
                got[x] += g[x] / 400
            else:
                r = np.maximum(p - g, 0)
                got += g[x] / 400 * r / r.sum()
                draws = [so.accept_sequence(z, [g, g], [0, x], [-1, 0], [0, u], v, 1.0)[1]
                         for v in (0.01, 0.99)]
                assert draws == [int(np.argmax(np.cumsum(r) > v * r.sum())) for v in (0.01, 0.99)]
    assert np.abs(got - p).max() < 4 / 400  # one grid step of u per token


def test_siblings_drawn_from_one_distribution_leave_the_target_distribution():
    z = np.array([[0.9, -0.4, 0.1]] * 3)
    p = _softmax(z[0])
    g = np.array([0.2, 0.5, 0.3])
    grid = (np.arange(60) + 0.5) / 60
    got = np.zeros(3)
    for x, y in itertools.product(range(3), range(3)):
        for u1, u2 in itertools.product(grid, grid):
            path, _, _ = so.accept_sequence(z, [g] * 3, [0, x, y], [-1, 0, 0], [0, u1, u2], 0.5, 1.0)
            w = g[x] * g[y] / 3600
            if len(path) == 2:
                got[x if path[1] == 1 else y] += w
            else:
                r = np.maximum(p - g, 0)
                r = np.maximum(r / r.sum() - g, 0)
                got += w * r / r.sum()
    assert np.abs(got - p).max() < 3 / 60


def test_proposals_without_probabilities():
    z = np.log(np.array([[0.5, 0.3, 0.2], [0.1, 0.1, 0.8], [1.0, 1.0, 1.0]]))
    par = [-1, 0, 0]
    # Child 1 proposes token 0 (taken iff u < 0.5), child 2 token 1 (iff u < 0.3 / 0.5).
    f = lambda u1, u2, v: so.accept_sequence(z, None, [9, 0, 1], par, [0, u1, u2], v, 1.0)[:2]  # noqa: E731
    assert f(0.49, 0.0, 0.95) == ([0, 1], 2)
    assert f(0.51, 0.59, 0.5) == ([0, 2], 1)
    assert f(0.51, 0.61, 0.0) == ([0], 2)      # only token 2 is left
    # The same token twice: the second proposal cannot be taken.
    assert so.accept_sequence(z, None, [9, 0, 0], par, [0, .6, 0.0], 0.0, 1.0)[:2] == ([0], 1)


def test_greedy_takes_the_lowest_index_of_the_maximum():
    z = np.array([[1.0, 3.0, 3.0], [2.0, 2.0, 0.0], [0.0, 0.0, 5.0]])
    assert so.accept_sequence(z, None, [7, 1, 0], [-1, 0, 1], [0, .99, .99], 0.7, 0.0)[:2] == ([0, 1, 2], 2)
    assert so.accept_sequence(z, None, [7, 2, 0], [-1, 0, 1], [0, 0, 0], 0.7, 0.0)[:2] == ([0], 1)


@pytest.mark.parametrize("row", [[np.nan, 0, 0], [np.inf, 0, 0], [-np.inf] * 3])
def test_a_row_without_distribution_ends_the_path(row):
    z = np.array([[0.0, 5.0, 0.0], row, [0.0, 0.0, 0.0]])
    assert so.accept_sequence(z, None, [0, 1, 1], [-1, 0, 1], [0, 0, 0], 0.5, 1.0)[:2] == ([0, 1], -1)


def test_fork_shares_full_pages_and_copies_the_partial_one():
    t = np.array([[5, 2, 7, -1], [-1] * 4, [3, -1, -1, -1]])
    ref = np.array([0, 0, 1, 1, 0, 1, 0, 1])
    t2, r2, copies, bad = so.pages_fork(t, ref, [0, 2], [1, 2], [33, 16], [4, 2])
    assert not bad and copies == [(7, 0)]
    assert t2.tolist() == [[5, 2, 7, -1], [5, 2, 0, 1], [3, 4, -1, -1]]
    assert r2.tolist() == [1, 1, 2, 1, 1, 2, 0, 1]
    assert so.pages_fork(t, ref, [0], [1], [33], [2])[3] == {"overflow"}
    assert so.pages_fork(t, ref, [0, 0], [1, 1], [3, 3], [1, 1])[3] == {"rows"}
    assert so.pages_fork(t, ref, [1], [2], [3], [1])[3] == {"block"}
    t4, r4, c4, bad = so.pages_fork(t, ref, [0] * 1, [1], [48], [3])
    assert not bad and c4 == [] and t4[1].tolist() == [5, 2, 7, -1]


def test_free_and_compact():
    t = np.array([[5, 2, 7, -1], [5, 2, 6, -1]])
    ref = np.array([0, 0, 2, 0, 0, 2, 1, 1])
    t2, r2, bad = so.pages_free(t, ref, [0, 0], [1, 2], [3, 4])
    assert not bad and t2[0].tolist() == [5, -1, -1, -1] and r2.tolist() == [0, 0, 1, 0, 0, 2, 1, 0]
    t3, r3, copies, live, bad = so.pages_compact(t2, r2)
    assert not bad and live == 3 and copies == [(5, 0), (6, 1)]
    assert t3.tolist() == [[0, -1, -1, -1], [0, 2, 1, -1]] and r3.tolist() == [2, 1, 1, 0, 0, 0, 0, 0]
