"""Oracle and binding of the caches in 4 bits, verification and eviction where calls meet:
no GPU."""

import numpy as np
import pytest
import torch

from host_transfer_gb300 import kv
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


# ---------------------------------------------------------------------------
# Binding


class Library:
    """Stands for the library: notes what was called."""

    def __init__(self):
        self.called = []

    def __getattr__(self, name):
        return lambda *args: self.called.append(name) or 0


@pytest.fixture
def library(monkeypatch):
    """Calls on CPU tensors, up to the library."""
    lib = Library()
    for name, stub in (("_load", lambda: lib), ("_for", lambda stream, device: (0, torch.enable_grad())),
                       ("_status", lambda status, device: 0), ("_on_device", lambda name, t: None), ("_checked", kv._Checked())):
        monkeypatch.setattr(kv, name, stub)
    return lib


def cache():
    return torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2, 16, 2), dtype=torch.bfloat16)


TABLE, LENS = torch.zeros((2, 2), dtype=torch.int32), torch.ones(2, dtype=torch.int32)


@pytest.mark.parametrize("which", ["k", "v", "k4", "v4"])
def test_a_store_refuses_what_requires_a_gradient(library, which):
    """What is read back from the cache would be attached to nothing, and no error reach the backward."""
    args = dict(k=torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16), v=torch.zeros((2, 1, 2, 64), dtype=torch.bfloat16),
                k4=cache(), v4=cache())
    kv.ibp_kv4_store(**args, table=TABLE, lens=LENS)
    (args[which][1] if "4" in which else args[which]).requires_grad_()
    with pytest.raises(ValueError, match="ibp_kv4_store.*detach"):
        kv.ibp_kv4_store(**args, table=TABLE, lens=LENS)
    assert library.called == ["ibp_kv4_store"]
    with torch.no_grad():
        kv.ibp_kv4_store(**args, table=TABLE, lens=LENS)
    assert library.called == ["ibp_kv4_store"] * 2


@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("which", ["q", "k", "lse", "weights"])
def test_weighing_in_place_refuses_what_requires_a_gradient(library, which, four):
    """It gives `weights` itself, not a view that the next step in place would refuse."""
    args = dict(q=torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16), k=cache() if four else torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16),
                lse=torch.zeros((2, 1, 4)), weights=torch.zeros((2, 32)))
    call = lambda inplace: kv.ibp_kv_weigh(**args, table=TABLE, lens=LENS, inplace=inplace)  # noqa: E731
    assert call(True) is args["weights"]
    (args[which][1] if isinstance(args[which], tuple) else args[which]).requires_grad_()
    n = len(library.called)
    with pytest.raises(ValueError, match="in place.*detach"):
        call(True)
    assert len(library.called) == n
    with torch.no_grad():
        assert call(True) is args["weights"]
    got = call(False)
    with pytest.raises(RuntimeError, match="no backward"):
        got.sum().backward()


@pytest.mark.parametrize("shape", [(2,), (2, 4, 8), (3, 32), ()])
def test_weights_of_another_shape_are_named(library, shape):
    """One dimension as long as the batch among them."""
    w = torch.zeros(shape)
    q, lse = torch.zeros((2, 1, 4, 64), dtype=torch.bfloat16), torch.zeros((2, 1, 4))
    for call in (lambda: kv.ibp_kv_weigh(q, cache(), TABLE, LENS, lse, w), lambda: kv.ibp_kv_evict(w, LENS, 4)):
        with pytest.raises(ValueError, match="weights must be a contiguous float32 tensor of shape .2, 'any'."):
            call()
    assert not library.called
    kv.ibp_kv_evict(torch.zeros((2, 32)), LENS, 4)
