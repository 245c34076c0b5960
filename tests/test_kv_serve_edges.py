"""Oracle and binding of the caches in 4 bits, verification and eviction where calls meet:
no GPU."""

import numpy as np

from oracle import kv_ref, kv_serve_ref as ref


def test_eviction_leaves_a_sequence_longer_than_its_weights_alone():
    """Seven tokens, six weights: three kept of the six that have one would be others of the seven."""
    w = np.array([[5, 1, 4, 2, 3, 0]], np.float32)
    path, n_draft, n_keep, out = ref.evict(w, [7], 3, 1, 1)
    assert path.tolist() == [[-1, -1, -1]] and n_draft.tolist() == n_keep.tolist() == [0] and np.array_equal(out, w)
    assert ref.evict(w, [6], 3, 1, 1)[0].tolist() == [[0, 2, 5]] and not ref.evict(w, [-1], 3, 1, 1)[3].any()
    pages = np.arange(8.0).reshape(1, 1, 8, 1)
    new, _, lens, _ = kv_ref.accept(pages, np.array([[0]]), np.array([7]), np.array([1]), n_draft, path, n_keep)
    assert np.array_equal(new, pages) and lens.tolist() == [7]


def test_acceptance_leaves_a_sequence_that_would_write_a_shared_page():
    """Pages 0 and 1 are both rows'; the first moves a token onto page 0, the second only onto its own page 2."""
    pages = np.arange(12.0).reshape(3, 1, 4, 1)
    args = np.array([[0, 1, -1], [0, 1, 2]]), np.array([8, 12]), np.array([2, 2, 1])
    new, table, lens, refs = kv_ref.accept(pages, *args, [8, 4], np.array([[0, 3, 5], [1, 2, -1]]), [3, 2])
    assert table.tolist() == args[0].tolist() and lens.tolist() == [8, 10] and refs.tolist() == [2, 2, 1]
    assert np.array_equal(new[:2], pages[:2]) and new[2].ravel().tolist() == [9, 10, 10, 11]
