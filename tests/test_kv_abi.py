"""The paged cache entry points without a GPU: scratch sizes, and refusals that come before any launch."""

import pytest
import torch

from host_transfer_gb300 import ibp, kv


@pytest.fixture(scope="module")
def lib():
    from host_transfer_gb300 import build

    build.build()
    return kv._load()


def test_scratch_sizes(lib):
    assert lib.ibp_kv_pages_workspace(100, 10) >= 4 * (100 + 2 * 10 + 1)
    assert lib.ibp_kv_pages_workspace(1 << 31, 0) > 1 << 32  # no 32-bit overflow
    # shapes that no call takes want nothing
    assert lib.ibp_tree_attention_workspace(1, 4, 16, 1, 8, 0, 64) == 0
    assert lib.ibp_tree_attention_workspace(1, 4, 16, 1, 7, 2, 64) == 0
    assert lib.ibp_tree_attention_workspace(1, 4, 0, 1, 8, 2, 64) == 0
    assert lib.ibp_sparse_attention_workspace(1, 4, 16, 1, 8, 2, 1024, 4) == 0
    # scores are kept only where there is a choice
    few = lib.ibp_sparse_attention_workspace(2, 64, 16, 1, 8, 2, 64, 64)
    many = lib.ibp_sparse_attention_workspace(2, 65, 16, 1, 8, 2, 64, 64)
    assert many >= few + 4 * 2 * 2 * 65


def test_refusals_without_gpu(lib):
    assert lib.ibp_kv_fork(None, 16, None, 4, None, 1, None, None, None, None, None, None, 0, None, None) != ibp.IBP_OK
    assert lib.ibp_kv_copy(None, None, None, 1, None, None) != ibp.IBP_OK
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    for call in (lambda: kv.ibp_tree_attention(q, k, k, table, lens),
                 lambda: kv.ibp_kv_summarize(k, table, lens, torch.zeros((4, 2, 2, 64), dtype=torch.int8), torch.zeros((4, 2))),
                 lambda: kv.ibp_kv_fork(table, lens, lens, lens, 16),
                 lambda: kv.ibp_kv_compact(table, lens, 16),
                 lambda: kv.ibp_kv_copy(k, torch.zeros((1, 3), dtype=torch.int32), lens)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(ValueError, match="int32"):
        kv._ints("lens", lens.long(), 1)
    with pytest.raises(ValueError, match="any"):
        kv._ints("mask", table, 3, None)


def test_checks_are_kept_by_form_alone():
    """Two tensors of one form share an entry; nothing of their addresses is part of it."""
    a, b = torch.zeros((2, 3)), torch.ones((2, 3))
    assert kv._form(a) == kv._form(b) and kv._form(a) != kv._form(b.t()) and kv._form(None) is None
    calls = []
    for t in (a, b):
        kv._once(("form test", kv._form(t)), lambda: calls.append(1) or 7)
    assert calls == [1]
    for i in range(kv._MOST_CHECKED + 5):
        kv._once(("form test", i), lambda: i)
    assert len(kv._checked.calls) <= kv._MOST_CHECKED
