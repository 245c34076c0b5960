"""Hand-derived cases that pin the oracle of the paged cache operators."""

import numpy as np
import pytest

from oracle import kv_ref

I32 = np.int32


def test_fork_shares_full_pages_and_copies_the_last_one():
    # page of 4: row 0 holds 6 tokens (pages 5, 2), row 1 holds 4 (page 0)
    table = np.array([[5, 2, -1], [0, -1, -1]], I32)
    refs = np.array([1, 0, 1, 0, 0, 1], I32)
    out, lens, refs, moves, short = kv_ref.fork(table, np.array([6, 4], I32), refs, [0, 0, 0], 4)
    # row 1 had no child: page 0 is free and serves the first copy
    assert out.tolist() == [[5, 2, -1], [5, 0, -1], [5, 1, -1]]
    assert lens.tolist() == [6, 6, 6] and refs.tolist() == [1, 1, 1, 0, 0, 3]
    assert moves == [(2, 0, 2), (2, 1, 2)] and not short


def test_fork_without_a_free_page_keeps_the_full_pages():
    table = np.array([[0, 1]], I32)
    out, lens, refs, moves, short = kv_ref.fork(table, np.array([5], I32), np.array([1, 1], I32), [0, 0], 4)
    assert short and lens.tolist() == [5, 4] and out.tolist() == [[0, 1], [0, -1]]
    assert refs.tolist() == [2, 1] and moves == []


def test_free_and_compact():
    table = np.array([[4, 1], [3, -1], [5, 4]], I32)
    refs = np.array([0, 1, 0, 1, 2, 1], I32)
    table, lens, refs = kv_ref.free(table, np.array([8, 2, 8], I32), refs, [0], 4)
    assert refs.tolist() == [0, 0, 0, 1, 1, 1] and lens.tolist() == [0, 2, 8]
    table, refs, moves = kv_ref.compact(table, refs, 4)
    assert moves == [(3, 0, 4), (4, 1, 4), (5, 2, 4)]
    assert table.tolist() == [[-1, -1], [0, -1], [2, 1]] and refs.tolist() == [1, 1, 1, 0, 0, 0]


def test_accept_moves_rows_and_frees_pages():
    pool = np.arange(12.0).reshape(1, 6, 1, 2, 1)  # pages of 2 tokens
    table = np.array([[3, 0, 5]], I32)
    refs = np.array([1, 0, 0, 1, 0, 1], I32)
    # 6 tokens, the last 4 drafted: tokens 1 and 3 of them are kept at positions 2 and 3
    new, table, lens, refs = kv_ref.accept(pool, table, np.array([6], I32), refs, [4], np.array([[1, 3]]), [2])
    assert lens.tolist() == [4] and table.tolist() == [[3, 0, -1]] and refs.tolist() == [1, 0, 0, 1, 0, 0]
    assert new[0, 0, 0, :, 0].tolist() == [1.0, 11.0]


def test_attention_of_equal_scores_is_the_mean():
    k = np.zeros((2, 1, 2, 4))
    v = np.arange(16.0).reshape(2, 1, 2, 4)
    q = np.ones((1, 2, 1, 4))
    table, lens = np.array([[1, 0]], I32), np.array([4], I32)
    out, lse, _, _ = kv_ref.tree_attention(q, k, v, table, lens)
    # token 0 of the draft sees positions 0, 1 (page 1) and itself; token 1 sees all four
    assert np.allclose(out[0, 0, 0], (v[1, 0, 0] + v[1, 0, 1] + v[0, 0, 0]) / 3)
    assert np.allclose(out[0, 1, 0], v.reshape(4, 4).mean(0)) and np.allclose(lse[0, :, 0], np.log([3, 4]))
    out, lse, _, _ = kv_ref.tree_attention(q, k, v, table, lens, mask=np.array([[[0], [1]]]))
    assert np.allclose(lse[0, :, 0], np.log([2, 3]))
    out, lse, _, _ = kv_ref.tree_attention(q, k, v, table, np.array([2], I32), mask=np.array([[[0], [2]]]))
    assert not out[0, 0].any() and lse[0, 0, 0] == -np.inf and np.allclose(out[0, 1, 0], v[1, 0, 1])


def test_bounds_of_a_page():
    k = np.array([[[[1.0, -2.0], [0.5, 4.0], [100.0, 100.0]]]], np.float32)
    codes, scales = kv_ref.summarize(k, np.array([[0]], I32), np.array([2], I32), np.zeros((1, 1, 2, 2), np.int8),
                                     np.zeros((1, 1), np.float32))
    # a = 4: 127/4 = 31.75 a unit; the third token is not valid
    assert codes[0, 0].tolist() == [[16, -64], [32, 127]] and scales[0, 0] == pytest.approx(4 / 127)


def test_selection_takes_forced_pages_then_the_highest_bounds():
    codes = np.zeros((5, 2, 1), np.int8)
    codes[:, 1, 0] = [9, 3, 7, 7, 1]
    scales = np.ones(5, np.float32)
    table = np.arange(5)
    q = np.ones((1, 1), np.float32)
    pick = lambda *a: kv_ref.select(q, codes, scales, table, 9, 2, *a)  # noqa: E731
    assert pick(2, 0, 1) == [0, 4]
    assert pick(3, 1, 1) == [0, 2, 4]  # pages 2 and 3 tie: the lower one
    assert pick(4, 0, 2) == [0, 2, 3, 4]
    assert pick(5, 0, 1) == [0, 1, 2, 3, 4]
    assert kv_ref.select(-q, codes, scales, table, 9, 2, 2, 0, 1) == [0, 4]  # minima are all 0: the lowest page


def test_a_page_of_infinite_scale_comes_first():
    codes = np.ones((4, 2, 1), np.int8)
    scales = np.array([1, 1, np.inf, 1], np.float32)
    assert kv_ref.select(np.ones((1, 1), np.float32), codes, scales, np.arange(4), 7, 2, 2, 0, 1) == [2, 3]
