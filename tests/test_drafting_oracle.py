"""The references of oracle/drafting_ref.py, pinned by hand-made examples and by
the references that they extend."""
import math

import numpy as np

from oracle import drafting_ref as ref
from oracle import serving_ref


def test_one_axis_is_the_plain_rotation():
    rng = np.random.default_rng(1)
    x, table = rng.normal(size=(2, 3, 5, 24)), rng.normal(size=(9, 16))
    pos = rng.integers(-1, 9, size=(2, 5))
    for inter in (False, True):
        for inverse in (False, True):
            a = ref.rope_axes(x, pos[None], table, [0] * 8, 4, inter, inverse)
            b = serving_ref.rope(x, pos, table, 4, inter, inverse)
            np.testing.assert_allclose(a, b, rtol=0, atol=1e-15)


def test_axes_by_hand():
    """Two pairs, quarter turns for axis 0 and half turns for axis 1."""
    table = np.array([[1, 1, 0, 0], [0, -1, 1, 0]], dtype=float)  # cos | sin of positions 0, 1
    x = np.array([1.0, 2.0, 3.0, 4.0]).reshape(1, 1, 1, 4)
    one = np.ones((1, 1), dtype=int)
    y = ref.rope_axes(x, np.stack([one, one]), table, [0, 1])
    np.testing.assert_allclose(y.ravel(), [-3, -2, 1, -4])  # (1, 3) by 90 degrees, (2, 4) by 180
    y = ref.rope_axes(x, np.stack([0 * one, one]), table, [0, 1])
    np.testing.assert_allclose(y.ravel(), [1, -2, 3, -4])
    y = ref.rope_axes(y, np.stack([0 * one, one]), table, [0, 1], inverse=True)
    np.testing.assert_allclose(y, x)


def test_tree_keys_by_hand():
    #   context 0 1 2, tokens in the slots 3 .. 7:  0 -> (1, 2 -> 4), 3 a second root
    keys = ref.tree_keys([-1, 0, 0, -1, 2], 8)
    assert [k for k, _ in keys] == [[0, 1, 2, 3], [0, 1, 2, 3, 4], [0, 1, 2, 3, 5], [0, 1, 2, 6], [0, 1, 2, 3, 5, 7]]
    assert [d for _, d in keys] == [0, 1, 1, 0, 2]
    # a window of 2 keys before a token: positions 3, 4, 4, 3, 5
    keys = ref.tree_keys([-1, 0, 0, -1, 2], 8, 2)
    assert [k for k, _ in keys] == [[1, 2, 3], [2, 3, 4], [2, 3, 5], [1, 2, 6], [3, 5, 7]]
    keys = ref.tree_keys([-1, 0, 0, -1, 2], 8, 0)
    assert [k for k, _ in keys] == [[3], [4], [5], [6], [7]]
    # padding, its descendants, parents that are no earlier token, and slots before the sequence
    assert [k for k, _ in ref.tree_keys([-2, 0, 2, -1, 3], 6)] == [[], [], [], [0, 4], [0, 4, 5]]
    assert [k for k, _ in ref.tree_keys([-1, -1, 0, 1], 3)] == [[], [0], [], [0, 2]]
    assert [k for k, _ in ref.tree_keys([-1, -1], 0)] == [[], []]


def test_a_chain_is_the_plain_decode():
    rng = np.random.default_rng(2)
    q, k, v = rng.normal(size=(2, 4, 3, 8)), rng.normal(size=(6, 2, 4, 8)), rng.normal(size=(6, 2, 4, 5))
    bt, lens, chain = [[0, 3, 5], [2, 1, 4]], [11, 7], [[-1, 0, 1]] * 2
    for window in (-1, 0, 4):
        a = ref.tree_decode(q, k, v, bt, lens, chain, 0.4, 3.0, window, [0.5, 2.0], [1.5, 1.0])
        b = serving_ref.decode(q, k, v, bt, lens, 0.4, 3.0, window, [0.5, 2.0], [1.5, 1.0])
        # (sums of a dozen terms of size 1 in another order: each off by some 2^-53 of the terms, however small the sum)
        for x, y in zip(a, b):
            np.testing.assert_allclose(x, y, rtol=1e-13, atol=1e-14)


def test_empty_rows():
    q = np.ones((1, 1, 2, 4))
    c = np.ones((1, 1, 4, 4))
    out, lse, _, _ = ref.tree_decode(q, c, c, [[0]], [3], [[-2, -1]], 1.0)
    assert (out[0, 0, 0] == 0).all() and lse[0, 0, 0] == -math.inf and math.isfinite(lse[0, 0, 1])


def test_compact_by_hand():
    cache = np.arange(12.0).reshape(3, 1, 4, 1)
    got = ref.compact(cache, [[2, 0]], [[1, 4, 6, -1, 7]], [0])  # tokens 9, 0, 2 to the front
    assert got[2, 0, :, 0].tolist() == [9, 0, 2, 11] and got[:2].tolist() == cache[:2].tolist()


def test_remap_by_hand():
    # one row of 10 tokens (pages 5, 3, 7 of 4 rows), page 0 held by someone else
    table, refs = [[5, 3, 7, -1]], [1, 0, 0, 1, 0, 1, 0, 1]
    # three heirs: two continue all of it, one the first 6 tokens; a fourth is new
    new, out, copies, short = ref.remap(table, [0, 0, 0, -1], [10, 10, 6, 0], [13, 10, 6, 3], refs, 4)
    assert new == [[5, 3, 7, 1], [5, 3, 2, -1], [5, 4, -1, -1], [6, -1, -1, -1]]
    assert copies == [[-1, -1, 0], [7, 2, 2], [3, 4, 2], [-1, -1, 0]] and short == 0
    assert out == [1, 1, 1, 2, 1, 3, 1, 1]
    # nobody goes on: all of its pages are free
    assert ref.remap(table, [-1], [0], [0], refs, 4)[1] == [1, 0, 0, 0, 0, 0, 0, 0]
    # a roll back within its own last page: nothing is copied
    assert ref.remap(table, [0], [9], [9], refs, 4)[0] == [[5, 3, 7, -1]]
    # five pages wanted of four
    new, out, copies, short = ref.remap(table, [0, 0, -1], [10, 10, 0], [16, 12, 12], refs, 4)
    assert short == 1 and new[2] == [4, 6, -1, -1]
    # a last page that someone else holds too is copied
    new, _, copies, _ = ref.remap(table, [0], [9], [9], [0, 0, 0, 1, 0, 1, 0, 2], 4)
    assert new == [[5, 3, 0, -1]] and copies == [[7, 0, 1]]


def test_copy_by_hand():
    cache = np.arange(12.0).reshape(3, 1, 4, 1)
    got = ref.copy(cache, [[0, 2, 3], [-1, -1, 0], [1, 0, 0]])
    assert got[2, 0, :, 0].tolist() == [0, 1, 2, 11] and got[:2].tolist() == cache[:2].tolist()
