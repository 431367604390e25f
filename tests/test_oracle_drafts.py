"""Pins of the oracle for drafted tokens: the norm's length, a tree's rows against whole sequences of
their own, and the verification's distribution by counting every outcome."""
import itertools

import numpy as np

from oracle import drafts as O
from oracle import mixers as M


def test_norm_has_unit_mean_square_and_scales():
    x = np.random.default_rng(1).standard_normal((3, 4, 64))
    y = O.norm(x, np.ones(64), 0.0)
    assert np.allclose((y ** 2).mean(-1), 1) and np.allclose(O.norm(7 * x, np.ones(64), 0.0), y)
    w = np.arange(64.0)
    assert np.allclose(O.norm(x, w, 0.1), x * w / np.sqrt((x ** 2).mean(-1, keepdims=True) + 0.1))
    assert (O.norm(np.zeros((1, 64)), w, 0.0) == 0).all()


def test_ways():
    tree = [-1, 0, 0, 2, -1, 4, 9, 6, -3, 7]
    assert [O.way(tree, i) for i in range(10)] == [[0], [0, 1], [0, 2], [0, 2, 3], [4], [4, 5], [], [], [], []]
    assert O.way(None, 3) == [0, 1, 2, 3]
    assert list(O.seen(tree, 3, 2, 0)) == [0, 1, 2, 4, 5] and list(O.seen(tree, 3, 2, 4)) == [1, 2, 4, 5]
    assert list(O.seen(tree, 3, 2, 2)) == [4, 5] and list(O.seen(tree, 6, 2, 0)) == []


def test_a_nodes_rows_are_those_of_its_own_sequence():
    """Attention of a node equals that of one token at the end of the sequence its way makes."""
    rng = np.random.default_rng(2)
    tree, ctx, W, H, D = np.array([[-1, 0, 0, 1, 2, -2]]), 19, 6, 4, 16
    k, v = rng.standard_normal((2, 4, 8, 2, D))
    table, q = np.array([[3, 0, 2, 1]]), rng.standard_normal((1, W, H, D))
    for window in (0, 3, 10):
        out, lse, mag, _ = O.attend(q, k, v, table, [ctx], tree, 20, 0.4, window, 2)
        for i in range(W):
            rows = list(range(ctx)) + [ctx + j for j in O.way(tree[0], i)]
            if len(rows) == ctx:
                assert (out[0, i] == 0).all() and np.isneginf(lse[0, i]).all()
                continue
            pool = [np.zeros((4, 8, 2, D)) for _ in range(2)]
            for n, r in enumerate(rows):
                for p, src in zip(pool, (k, v)):
                    p[n // 8, n % 8] = src[table[0, r // 8], r % 8]
            ref, rl, _, _ = M.attend(q[:, i], *pool, np.arange(4)[None], [len(rows)], 32, 0.4, window, 2)
            assert np.allclose(out[0, i], ref[0]) and np.allclose(lse[0, i], rl[0])
    assert (mag >= 0).all()


def _outcomes(logits, drafts, parents, t, draft, steps=24):
    """Frequencies of the first emitted token over a grid of all uniform numbers it depends on."""
    W, V = logits.shape
    seen = np.zeros(V)
    grid = (np.arange(steps) + 0.5) / steps
    for u in itertools.product(grid, repeat=2):             # node 0's number and the last one's
        uniforms = np.full(W + 1, 0.5)
        uniforms[0], uniforms[W] = u
        seen[O.verify(logits, drafts, parents, t, uniforms, draft)[0][0]] += 1
    return seen / steps ** 2


def test_first_token_has_the_targets_distribution():
    rng = np.random.default_rng(3)
    logits, draft = rng.standard_normal((2, 4, 5)).astype(np.float32)
    p = O.softmax(logits[0], 0.8)
    got = _outcomes(logits, [0, 2, 2, 4], [-1, 0, 0, 0], 0.8, None)
    assert np.abs(got - p).max() < 0.06
    q = O.softmax(draft[0], 0.8)                            # drawn drafts: average over what was drawn
    got = sum(q[x] * _outcomes(logits, [0, x, 1, 1], None, 0.8, draft) for x in range(5))
    assert np.abs(got - p).max() < 0.06


def test_walks():
    logits = np.full((4, 6), -np.inf, np.float32)
    for i, t in enumerate([2, 4, 1, 5]):
        logits[i, t] = 0
    tree = [-1, 0, 0, 2]
    assert O.verify(logits, [0, 3, 2, 1], tree, 0, None)[:2] == ([2, 1, 5], [0, 2, 3])
    assert O.verify(logits, [0, 2, 2, 1], tree, 0, None)[:2] == ([2, 4], [0, 1])
    assert O.verify(logits, [0, 3, 2, 1], tree, 1.0, np.full(5, 0.99))[:2] == ([2, 1, 5], [0, 2, 3])
    assert O.verify(logits, [0, 3, 3, 1], tree, 1.0, np.full(5, 0.5))[:2] == ([2], [0])
    assert O.verify(logits, [0, 3, 3, 1], [-2, 0, 0, 2], 1.0, np.full(5, 0.5))[:2] == ([], [])


def test_compact_and_copy():
    pool = np.arange(4 * 4).reshape(4, 4, 1).copy()
    O.compact([pool], np.array([[2, 0, 3]]), [3], np.array([[0, 2, 3, 1]]), [4])
    # rows 3 .. 6 of the sequence are (2,3), (0,0), (0,1), (0,2)
    assert pool[2, 3] == 11 and list(pool[0, :, 0]) == [1, 2, 0, 3]
    O.copy_pages([pool], [0, 9], [1, 2])
    assert (pool[1] == pool[0]).all() and pool[2, 3] == 11
