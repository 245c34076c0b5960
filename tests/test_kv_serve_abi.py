"""The caches in 4 bits, verification and eviction without a GPU: scratch sizes,
constants, and refusals that come before any launch."""

import ctypes
import os
import re

import pytest
import torch

from host_transfer_gb300 import ibp, kv

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "ibp.h")


@pytest.fixture(scope="module")
def lib():
    from host_transfer_gb300 import build

    build.build()
    return kv._load()


def test_constants_are_the_headers():
    text = open(HEADER).read()
    for name in ("IBP_KV4_GROUP", "IBP_VERIFY_MAX_VOCAB", "IBP_VERIFY_MAX_DRAFT"):
        assert getattr(kv, name) == int(re.search(rf"#define {name} (\d+)u", text).group(1))


def test_the_structure_is_the_headers():
    """Every field of ibp_kv4_pages, in order, with its size."""
    text = open(HEADER).read()
    body = re.sub(r"/\*.*?\*/", "", re.search(r"typedef struct ibp_kv4_pages \{(.*?)\} ibp_kv4_pages;", text, re.S).group(1), flags=re.S)
    sizes = {"void*": 8, "int64_t": 8, "uint64_t": 8, "uint32_t": 4}
    want = []
    for line in filter(None, (x.strip() for x in body.split(";"))):
        kind, names = line.split(None, 1)
        want += [(n.strip(), sizes[kind]) for n in names.split(",")]
    assert [(n, ctypes.sizeof(t)) for n, t in kv._Pages4._fields_] == want


def test_scratch_sizes(lib):
    size = lib.ibp_kv4_attention_workspace
    # shapes that no call takes want nothing
    assert size(1, 4, 16, 1, 8, 0, 64) == size(1, 4, 16, 1, 7, 2, 64) == size(1, 4, 0, 1, 8, 2, 64) == size(1, 4, 16, 1, 8, 2, 288) == 0
    assert size(1, 4, 16, 1, 8, 2, 64) < 1 << 16  # a part of each of a few blocks
    assert size(64, 1024, 64, 1, 64, 8, 128) < 1 << 30  # parts of the blocks that the GPU holds at once
    # many rows decode the cache once, but not one of more than 4 GB
    assert size(4, 256, 64, 1024, 8, 8, 128) > 4 * 256 * 64 * 8 * 128 * 4
    assert size(64, 4096, 64, 1024, 8, 8, 128) < 1 << 30


def test_refusals_without_gpu(lib):
    assert lib.ibp_kv_evict(None, 8, None, 1, 4, 1, 1, None, None, None, None, None, None) != ibp.IBP_OK
    assert lib.ibp_kv_verify(None, 0, 0, None, 0, 0, 8, None, None, None, 1, 1, None, None, None, None, None, None) != ibp.IBP_OK
    k4 = torch.zeros((4, 2, 16, 32), dtype=torch.uint8), torch.zeros((4, 2, 16, 2), dtype=torch.bfloat16)
    table, lens = torch.zeros((1, 2), dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16)
    p, u, w = torch.zeros((1, 2, 9)), torch.zeros((1, 2)), torch.zeros((1, 32))
    for call in (lambda: kv.ibp_kv4_store(q[:, :, :2], q[:, :, :2], k4, k4, table, lens),
                 lambda: kv.ibp_kv4_load(k4, k4, table, lens, 1),
                 lambda: kv.ibp_kv4_attention(q, k4, k4, table, lens),
                 lambda: kv.ibp_kv_weigh(q, k4, table, lens, torch.zeros((1, 1, 4)), w),
                 lambda: kv.ibp_kv_verify(p, lens[None], u),
                 lambda: kv.ibp_kv_evict(w, lens, 4)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for kw in (dict(budget=0), dict(budget=4, keep_first=5), dict(budget=4, keep_last=-1), dict(budget=1 << 31)):
        with pytest.raises(ValueError, match="budget"):
            kv.ibp_kv_evict(w, lens, **kw)


def test_a_gradient_for_attention_is_an_error():
    q, out, lse = torch.randn(2, 3, requires_grad=True), torch.randn(2, 3), torch.randn(2)
    got = kv._results("ibp_kv4_attention", out, lse, q, out, out)
    with pytest.raises(RuntimeError, match="ibp_kv4_attention has no backward"):
        got[0].sum().backward()
