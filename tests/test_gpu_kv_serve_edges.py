"""GPU tests of the calls around the caches in 4 bits, verification and eviction that
hand one's results to the next, and of their less usual layouts, against the CPU oracle."""

import numpy as np
import pytest
import torch

from host_transfer_gb300 import ibp, kv
from oracle import kv_ref, kv_serve_ref as ref
from tests.kv_util import dev, host, tables
from tests.test_gpu_kv_serve import gen

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    yield
    assert kv.ibp_kv_get_status(raise_on_error=False) == ibp.IBP_OK


def err(code):
    """The status the test has provoked, read and cleared."""
    assert kv.ibp_kv_get_status(raise_on_error=False) == code


# ---------------------------------------------------------------------------
# Eviction and the move that follows from it


@pytest.mark.parametrize("width,budget", [(30, 10), (9001, 4), (40, 64)])
def test_a_sequence_longer_than_its_weights_is_left_alone(width, budget):
    """What the choice gives goes to ibp_kv_accept with the true lengths: a sequence whose
    tokens do not all have a weight keeps every one of them, where it was."""
    rng = np.random.default_rng(width)
    lens = np.array([width + 1, width, width + 33, width - 7, 3], np.int32)
    w = rng.random((len(lens), width)).astype(np.float32)
    want = ref.evict(w, lens, budget, 1, 1)
    got = kv.ibp_kv_evict(dev(w, torch.float32), dev(lens), budget, keep_first=1, keep_last=1)
    err(ibp.IBP_ERANGE)
    for x, y, name in zip(got, want, ("path", "n_draft", "n_keep", "weights")):
        assert np.array_equal(host(x), y), name
    for b in (0, 2):
        assert want[1][b] == want[2][b] == 0 and (want[0][b] == -1).all() and np.array_equal(want[3][b], w[b])
    page = 16
    table, refs = tables(lens, page, int((-(-lens // page)).sum()) + 2, -(-int(lens.max()) // page), rng)
    pages = torch.randn((len(refs), 2, page, 8), device="cuda", generator=gen(1)).bfloat16()
    moved = kv_ref.accept(host(pages), table, lens, refs, want[1], want[0], want[2])
    after = kv.ibp_kv_accept(pages, dev(table), dev(lens), dev(refs), got[1], got[0], got[2])
    assert np.array_equal(host(pages), moved[0])
    assert all(np.array_equal(host(x), y) for x, y in zip(after, moved[1:]))
    assert host(after[1])[0] == width + 1 and host(after[1])[2] == width + 33
