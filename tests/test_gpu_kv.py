"""GPU tests of the paged key/value cache operators against the CPU oracle."""

import ctypes
import math
import random

import numpy as np
import pytest
import torch

from host_transfer_gb300 import ibp, kv
from oracle import kv_ref
from tests.kv_util import DTYPES, check_attention, dev, host, poison, pool, tables

pytestmark = pytest.mark.gpu

LAYOUTS = ["hnd", "nhd", "padded"]


@pytest.fixture(autouse=True)
def clean_status():
    yield
    assert kv.ibp_kv_get_status(raise_on_error=False) == ibp.IBP_OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def err(code):
    """The status the test has provoked, read and cleared."""
    assert kv.ibp_kv_get_status(raise_on_error=False) == code


# ---------------------------------------------------------------------------
# Pages


def moves_of(moves, count):
    n = int(count.item())
    m = host(moves)
    assert (m[n:] == -1).all()
    return [tuple(int(x) for x in r) for r in m[:n]]


def shared_state(rng, n_seqs, page, longest, n_pages):
    lens = rng.integers(0, longest + 1, n_seqs)
    table, refs = tables(lens, page, n_pages, -(-longest // page) + 1, rng)
    return table, lens.astype(np.int32), refs


@pytest.mark.parametrize("n_seqs,n_out,page,longest,n_pages", [
    (1, 1, 16, 40, 8), (1, 5, 16, 40, 8), (4, 4, 16, 0, 3), (3, 40, 1, 9, 40), (7, 64, 64, 500, 120),
    (30, 700, 24, 100, 900), (64, 2000, 16, 60, 5000), (5, 0, 16, 40, 20),
    (64, 4000, 16, 60, 20000), (300, 300, 16, 900, 30000),  # a cluster of CTAs
])
def test_fork(n_seqs, n_out, page, longest, n_pages):
    rng = np.random.default_rng(n_seqs * 1000 + n_out)
    table, lens, refs = shared_state(rng, n_seqs, page, longest, n_pages)
    parents = rng.integers(0, n_seqs, n_out).astype(np.int32)
    want = kv_ref.fork(table, lens, refs, parents.tolist(), page)
    got = kv.ibp_kv_fork(dev(table), dev(lens), dev(refs), dev(parents), page)
    assert np.array_equal(host(got[0]), want[0]) and np.array_equal(host(got[1]), want[1])
    assert np.array_equal(host(got[2]), want[2])
    assert moves_of(got[3], got[4]) == want[3]
    err(ibp.IBP_ENOMEM if want[4] else ibp.IBP_OK)
    # a second generation: the children share pages with one another
    if n_out and not want[4]:
        again = rng.integers(0, n_out, n_out).astype(np.int32)
        w2 = kv_ref.fork(*want[:3], again.tolist(), page)
        g2 = kv.ibp_kv_fork(*got[:3], dev(again), page)
        assert all(np.array_equal(host(g2[i]), w2[i]) for i in range(3)) and moves_of(*g2[3:]) == w2[3]
        err(ibp.IBP_ENOMEM if w2[4] else ibp.IBP_OK)


def test_fork_out_of_pages():
    rng = np.random.default_rng(3)
    table, refs = tables([70, 20], 16, 9, 6, rng)
    lens = np.array([70, 20], np.int32)
    parents = [0, 0, 1, 1, 0, 1]
    want = kv_ref.fork(table, lens, refs, parents, 16)
    assert want[4]
    got = kv.ibp_kv_fork(dev(table), dev(lens), dev(refs), dev(np.array(parents)), 16)
    assert all(np.array_equal(host(got[i]), want[i]) for i in range(3)) and moves_of(*got[3:]) == want[3]
    err(ibp.IBP_ENOMEM)


def test_fork_bad_rows_are_empty():
    rng = np.random.default_rng(4)
    table, refs = tables([20], 16, 6, 3, rng)
    got = kv.ibp_kv_fork(dev(table), dev(np.array([20])), dev(refs), dev(np.array([0, 7, -1])), 16)
    assert host(got[1]).tolist() == [20, 0, 0] and (host(got[0])[1:] == -1).all()
    assert np.array_equal(host(got[2]), refs)
    err(ibp.IBP_ERANGE)


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("n_seqs,page,longest,n_pages", [(1, 16, 40, 8), (9, 64, 300, 60), (200, 16, 90, 3000),
                                                      (500, 16, 700, 40000)])
def test_free_and_compact(n_seqs, page, longest, n_pages, inplace):
    rng = np.random.default_rng(n_seqs)
    table, lens, refs = shared_state(rng, n_seqs, page, longest, n_pages)
    table, lens, refs, _, _ = kv_ref.fork(table, lens, refs, rng.integers(0, n_seqs, n_seqs).tolist(), page)
    gone = rng.permutation(n_seqs)[: n_seqs // 2]
    listed = np.concatenate([gone, gone[:1]]).astype(np.int32)  # a row listed twice is freed once
    w = kv_ref.free(table, lens, refs, listed.tolist(), page)
    g = kv.ibp_kv_free(dev(table), dev(lens), dev(refs), dev(listed), page, inplace=inplace)
    assert all(np.array_equal(host(a), b) for a, b in zip(g, w))
    w2 = kv_ref.compact(w[0], w[2], page)
    g2 = kv.ibp_kv_compact(g[0], g[2], page, inplace=inplace)
    assert np.array_equal(host(g2[0]), w2[0]) and np.array_equal(host(g2[1]), w2[1])
    assert moves_of(*g2[2:]) == w2[2]


@pytest.mark.parametrize("n", [1, 1000, 100001])
@pytest.mark.parametrize("live", ["none", "all", "last"])
def test_compact_extremes(live, n):
    refs = {"none": np.zeros(n), "all": np.ones(n), "last": (np.arange(n) == n - 1) * 3}[live].astype(np.int32)
    table = np.array([[n - 1, -1, n // 2]], np.int32)
    w = kv_ref.compact(table, refs, 8)
    g = kv.ibp_kv_compact(dev(table), dev(refs), 8)
    assert np.array_equal(host(g[0]), w[0]) and np.array_equal(host(g[1]), w[1]) and moves_of(*g[2:]) == w[2]


def test_free_reports_a_count_below_zero():
    got = kv.ibp_kv_free(dev(np.array([[0, 1]])), dev(np.array([20])), dev(np.array([1, 0])), dev(np.array([0])), 16)
    assert host(got[2]).tolist() == [0, 0]
    err(ibp.IBP_ECORRUPT)
    got = kv.ibp_kv_free(dev(np.array([[0, 9]])), dev(np.array([20])), dev(np.array([1, 0])), dev(np.array([0, 5])), 16)
    assert host(got[2]).tolist() == [0, 0]
    err(ibp.IBP_ERANGE)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("shape,dtype", [
    ((2, 9, 3, 16, 64), torch.bfloat16), ((1, 6, 1, 1, 8), torch.float16), ((4, 8, 2, 7, 5), torch.bfloat16),
    ((1, 7, 2, 5, 3), torch.int8), ((2, 5, 1, 64, 256), torch.float32), ((1, 6, 5, 1, 1), torch.float32),
    ((1, 5, 2, 3, 9), torch.float64),
])
def test_copy(shape, dtype, layout):
    g = gen(1)
    x = pool(shape, torch.float32, layout, g).mul(50)
    x = torch.empty_strided(x.shape, x.stride(), dtype=dtype, device="cuda").copy_(x.nan_to_num())
    moves = np.array([[0, 3, shape[3]], [1, 2, max(shape[3] - 1, 0)], [4, 4, 0]], np.int32)
    want = kv_ref.copy(x.cpu().to(torch.float64).numpy(), moves[:2].tolist())
    listed = np.concatenate([moves, np.full((2, 3), -1, np.int32)])
    kv.ibp_kv_copy(x, dev(listed), dev(np.array([3])))
    assert np.array_equal(x.cpu().to(torch.float64).numpy(), want)


def test_copy_skips_bad_ids_and_keeps_to_the_count():
    x = torch.arange(4 * 8, dtype=torch.float32, device="cuda").reshape(4, 1, 1, 8)
    before = x.clone()
    kv.ibp_kv_copy(x, dev(np.array([[0, 4, 1], [-1, 1, 1], [0, 1, 1]])), dev(np.array([2])))
    assert torch.equal(x, before)
    err(ibp.IBP_ERANGE)


def test_copy_past_32_bits():
    """A pool of more than 2^32 elements: offsets of its last pages need 64 bits."""
    n = 70000
    x = torch.zeros((n, 2, 32, 1024), dtype=torch.int8, device="cuda")
    x[n - 1] = 7
    x[n - 3] = 9
    kv.ibp_kv_copy(x, dev(np.array([[n - 1, 1, 32], [n - 3, n - 2, 32]])), dev(np.array([2])))
    assert (x[1] == 7).all() and (x[n - 2] == 9).all() and not x[2:100].any() and not x[0].any()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("pools,heads,page,dim,longest,draft", [
    (2, 3, 16, 64, 90, 24), (1, 1, 1, 8, 30, 12), (4, 2, 7, 5, 60, 40), (3, 2, 64, 128, 200, 1), (2, 2, 24, 80, 300, 200),
])
@pytest.mark.parametrize("inplace", [False, True])
def test_accept(pools, heads, page, dim, longest, draft, layout, inplace):
    rng = np.random.default_rng(draft)
    lens = rng.integers(draft, longest + 1, 6).astype(np.int32)
    table, refs = tables(lens, page, int((-(-lens // page)).sum()) + 2, -(-longest // page) + 2, rng)
    n_draft = np.array([draft, draft, 0, 1, max(draft // 2, 1), draft], np.int32)
    path = np.full((6, draft), -1, np.int32)
    n_accept = np.zeros(6, np.int32)
    for b in range(6):
        n_accept[b] = [rng.integers(0, n_draft[b] + 1), n_draft[b], 0, 1, n_draft[b] // 2, 0][b]
        path[b, : n_accept[b]] = np.sort(rng.permutation(n_draft[b])[: n_accept[b]])
    x = pool((pools, len(refs), heads, page, dim), torch.float16, layout, gen(2))
    want = kv_ref.accept(host(x), table, lens, refs, n_draft, path, n_accept)
    got = kv.ibp_kv_accept(x, dev(table), dev(lens), dev(refs), dev(n_draft), dev(path), dev(n_accept), inplace=inplace)
    assert np.array_equal(host(x), want[0])
    assert all(np.array_equal(host(a), b) for a, b in zip(got, want[1:]))


def test_accept_of_many_sequences():
    rng = np.random.default_rng(5)
    n, draft, page = 70, 20, 8
    lens = rng.integers(draft, 60, n).astype(np.int32)
    table, refs = tables(lens, page, 700, 8, rng)
    n_draft, n_accept = np.full(n, draft, np.int32), rng.integers(0, draft + 1, n).astype(np.int32)
    path = np.sort(np.argsort(rng.random((n, draft)), 1).astype(np.int32), 1)
    for b in range(n):
        path[b, : n_accept[b]] = np.sort(rng.permutation(draft)[: n_accept[b]])
    x = pool((6, 700, 4, page, 64), torch.bfloat16, "nhd", gen(3))
    want = kv_ref.accept(host(x), table, lens, refs, n_draft, path, n_accept)
    got = kv.ibp_kv_accept(x, dev(table), dev(lens), dev(refs), dev(n_draft), dev(path), dev(n_accept))
    assert np.array_equal(host(x), want[0])
    assert all(np.array_equal(host(a), b) for a, b in zip(got, want[1:]))


def test_accept_stops_at_a_bad_path():
    x = torch.arange(8, dtype=torch.float32, device="cuda").reshape(1, 1, 8, 1)
    one = lambda *a: dev(np.array(a))  # noqa: E731
    got = kv.ibp_kv_accept(x, one([0]), one(8), one(1), one(4), one([1, 0, 3]), one(3))
    assert host(got[1]).tolist() == [5] and host(x).ravel().tolist() == [0, 1, 2, 3, 5, 5, 6, 7]
    err(ibp.IBP_ERANGE)
    got = kv.ibp_kv_accept(x, one([0]), one(8), one(1), one(9), one([1, 2, 3]), one(1))
    assert host(got[1]).tolist() == [8]
    err(ibp.IBP_ERANGE)


# ---------------------------------------------------------------------------
# Tree attention


def mask_words(sees):
    B, T, _ = sees.shape
    words = np.zeros((B, T, (T + 31) // 32), np.uint32)
    for i in range(T):
        words[:, :, i // 32] |= sees[:, :, i].astype(np.uint32) << np.uint32(i % 32)
    return words.view(np.int32)


def random_tree(rng, B, T):
    sees = np.zeros((B, T, T), bool)
    for b in range(B):
        for t in range(T):
            up = int(rng.integers(max(0, t - 8), t + 1)) - 1
            if up >= 0:
                sees[b, t] = sees[b, up]
            sees[b, t, t] = True
    return sees


def run_tree(dt, layout, lens, T, hk, G, page, D, mask="tree", n_draft=None, nan=True, seed=0, scale=None):
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    B, width = len(lens), max(1, -(-int(max(lens)) // page)) + 1
    n_pages = int((-(-lens // page)).sum()) + 3
    table, _ = tables(lens, page, n_pages, width, rng)
    g = gen(seed)
    k = pool((n_pages, hk, page, D), DTYPES[dt], layout, g)
    v = pool((n_pages, hk, page, D), DTYPES[dt], layout, g)
    if nan:  # what no sequence holds has no influence
        poison(k, table, lens)
        poison(v, table, lens, float("inf"))
    q = torch.randn((B, T, hk * G, D), device="cuda", generator=g).to(DTYPES[dt])
    words = mask_words(random_tree(rng, B, T)) if isinstance(mask, str) else mask
    got = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens), mask=None if words is None else dev(words),
                                n_draft=None if n_draft is None else dev(np.array(n_draft)), scale=scale)
    want = kv_ref.tree_attention(host(q), host(k), host(v), table, lens, words, n_draft, scale)
    check_attention(*got, *want, dt)
    return got


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lens,T,hk,G,page,D", [
    ([1], 1, 1, 1, 16, 64),                      # one token, one head
    ([777, 1, 16, 17], 1, 2, 4, 16, 128),        # single tokens, grouped heads
    ([33, 129, 250, 128], 5, 2, 7, 24, 80),      # odd group, pages that end inside a step
    ([40, 41, 300], 13, 3, 1, 64, 128),          # a tree of 13, no grouping
    ([70, 64, 333], 33, 1, 8, 32, 128),          # more rows than one tile, two mask words
    ([600], 64, 2, 8, 64, 128),
    ([520, 90], 20, 2, 2, 1, 40),                # one token a page
    ([100, 9], 9, 1, 3, 7, 8),
    ([150, 47], 3, 2, 5, 128, 256),              # the widest heads
    ([300, 260], 30, 1, 12, 16, 136),
    ([1025, 1024, 1023], 17, 1, 16, 128, 120),
    ([290], 257, 1, 2, 8, 96),                   # a draft longer than a tile
])
def test_tree_attention(lens, T, hk, G, page, D, layout, dt):
    run_tree(dt, layout, lens, T, hk, G, page, D)


@pytest.mark.parametrize("T,G,D,page", [(1, 1, 128, 16), (4, 2, 64, 20), (24, 8, 128, 64), (40, 8, 128, 128)])
def test_tree_attention_long(T, G, D, page):
    """Lengths that are split over many CTAs and joined."""
    run_tree("bf16", "hnd", [5000, T, 4097], T, 1, G, page, D, seed=5)


@pytest.mark.parametrize("T,G", [(6, 2), (48, 4)])
def test_tree_mask_kinds(T, G):
    rng = np.random.default_rng(1)
    run_tree("f16", "hnd", [60, T, 200], T, 2, G, 16, 64, mask=None)
    nothing = np.zeros((3, T, (T + 31) // 32), np.int32)
    got = run_tree("bf16", "hnd", [60, T, 200], T, 2, G, 16, 64, mask=nothing)
    assert (host(got[1])[1] == -np.inf).all()  # no context and nothing of the draft: empty rows
    dense = rng.integers(-2**31, 2**31, nothing.shape).astype(np.int32)  # any bits, those past the draft too
    run_tree("bf16", "nhd", [60, T, 200], T, 2, G, 16, 64, mask=dense)


@pytest.mark.parametrize("T,G", [(6, 2), (48, 4)])
def test_tree_ragged_drafts(T, G):
    run_tree("bf16", "hnd", [60, T, 200, 0, 9], T, 2, G, 16, 128, n_draft=[T, 3, 0, 0, 1])
    run_tree("f16", "hnd", [400, 300], T, 1, G, 64, 128, mask=None, n_draft=[1, T], scale=0.3)


@pytest.mark.parametrize("T,G,D", [(6, 2, 128), (48, 4, 64), (7, 1, 256)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_tree_masked_infinities_and_nan(T, G, D, dt):
    """Drafted tokens that hold infinities and NaN reach the rows that see them, and no other."""
    rng = np.random.default_rng(2)
    lens, page, hk = np.array([90], np.int32), 16, 1
    table, _ = tables(lens, page, 8, 7, rng)
    g = gen(3)
    k, v = (pool((8, hk, page, D), DTYPES[dt], "hnd", g) for _ in range(2))
    q = torch.randn((1, T, G, D), device="cuda", generator=g).to(DTYPES[dt])
    sees = random_tree(rng, 1, T)
    sees[0, :, 1] = False
    sees[0, 1, 1] = sees[0, 3, 1] = True
    sees[0, :, 2] = False
    sees[0, 2, 2] = True
    clean = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens), mask=dev(mask_words(sees)))
    at = lambda p: (int(table[0, p // page]), 0, p % page)  # noqa: E731
    ctx = 90 - T
    v[at(ctx + 1)][: D // 2] = float("inf")
    v[at(ctx + 1)][D // 2] = float("nan")
    k[at(ctx + 2)] = float("nan")
    out, lse = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens), mask=dev(mask_words(sees)))
    hit = np.zeros(T, bool)
    hit[[1, 3, 2]] = True
    assert torch.equal(out[0, ~torch.from_numpy(hit).cuda()], clean[0][0, ~torch.from_numpy(hit).cuda()])
    for t in (1, 3):
        assert (out[0, t, :, : D // 2] == float("inf")).all() and out[0, t, :, D // 2].isnan().all()
        assert torch.equal(out[0, t, :, D // 2 + 1 :], clean[0][0, t, :, D // 2 + 1 :])
    assert out[0, 2].isnan().all() and lse[0, 2].isnan().all()


@pytest.mark.parametrize("T,G", [(2, 4), (40, 4)])
def test_tree_large_scores(T, G):
    """Scores far apart: one key takes all, and masks of the type's lowest value in the keys."""
    run_tree("bf16", "hnd", [300, 77], T, 1, G, 16, 128, scale=40.0)
    run_tree("f16", "hnd", [300, 77], T, 1, G, 16, 128, scale=1e-4)


@pytest.mark.parametrize("T,G", [(2, 4), (40, 4)])
def test_tree_bad_pages_read_as_zeros(T, G):
    rng = np.random.default_rng(8)
    lens = np.array([200], np.int32)
    table, _ = tables(lens, 16, 20, 14, rng)
    table[0, 3], table[0, 5] = 20, -7
    g = gen(4)
    k, v = (pool((20, 1, 16, 64), torch.bfloat16, "hnd", g) for _ in range(2))
    q = torch.randn((1, T, G, 64), device="cuda", generator=g).bfloat16()
    got = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens))
    check_attention(*got, *kv_ref.tree_attention(host(q), host(k), host(v), table, lens), "bf16")
    err(ibp.IBP_ERANGE)
    # a draft longer than the sequence: positions before the first do not exist
    lens = np.array([T - 1], np.int32)
    got = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens))
    check_attention(*got, *kv_ref.tree_attention(host(q), host(k), host(v), table, lens), "bf16")
    err(ibp.IBP_ERANGE)


def test_tree_strided_queries_outputs_and_streams():
    g = gen(6)
    lens = np.array([100, 50], np.int32)
    table, _ = tables(lens, 16, 12, 8, np.random.default_rng(0))
    k, v = (pool((12, 2, 16, 64), torch.bfloat16, "hnd", g) for _ in range(2))
    wide = torch.randn((2, 4, 3, 8, 64), device="cuda", generator=g).bfloat16()
    q = wide[:, :, 1]  # a third of a fused projection
    want = kv.ibp_tree_attention(q.contiguous(), k, v, dev(table), dev(lens))
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    got = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens), out=out, lse=lse)
    assert got[0] is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    flip = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(kv.ibp_tree_attention(flip, k, v, dev(table), dev(lens))[0], want[0])
    side = torch.cuda.Stream()
    t, n = dev(table), dev(lens)
    torch.cuda.synchronize()
    got = kv.ibp_tree_attention(q, k, v, t, n, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kv.ibp_tree_attention(q, k, v, t, n)
    q.copy_(torch.randn(q.shape, device="cuda", generator=g))
    graph.replay()
    want = kv.ibp_tree_attention(q.contiguous(), k, v, t, n)
    assert torch.equal(got[0], want[0])


@pytest.mark.parametrize("T,G", [(3, 2), (33, 4)])
def test_tree_same_bits_every_time(T, G):
    a = run_tree("bf16", "hnd", [2000, 700], T, 2, G, 64, 128, seed=9)
    b = run_tree("bf16", "hnd", [2000, 700], T, 2, G, 64, 128, seed=9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("T,G", [(2, 2), (40, 2)])
def test_tree_pool_past_32_bits(T, G):
    """Pages whose offsets need more than 32 bits."""
    n, page, D = 70000, 256, 128
    k = torch.zeros((n, 1, page, D), dtype=torch.bfloat16, device="cuda")
    table = np.array([[n - 1, 3, n - 2]], np.int32)
    g = gen(1)
    for p in (n - 1, 3, n - 2):
        k[p].normal_(generator=g)
    q = torch.randn((1, T, G, D), device="cuda", generator=g).bfloat16()
    got = kv.ibp_tree_attention(q, k, k, dev(table), dev(np.array([600])))
    small, at = k[[n - 1, 3, n - 2]], np.array([[0, 1, 2]], np.int32)
    check_attention(*got, *kv_ref.tree_attention(host(q), host(small), host(small), at, np.array([600])), "bf16")


# ---------------------------------------------------------------------------
# Tree attention, enough work for the tensor-core kernel


def scratch_of(lens, T, hk, G, page, D):
    """Scratch of the call: the tensor-core kernel wants some, the few-row kernel here none."""
    width = max(1, -(-max(lens) // page)) + 1
    return kv._load().ibp_tree_attention_workspace(len(lens), width, page, T, hk * G, hk, D)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D,layout", [
    ([300, 17, 129], 4, 40, 4, 16, 128, "hnd"),      # one row tile, sequences in and between tiles
    ([250, 640], 7, 33, 3, 24, 80, "nhd"),           # pages that end inside a tile, odd group
    ([131, 1, 128], 1, 64, 16, 64, 64, "padded"),    # single tokens
    ([70, 200], 40, 12, 5, 8, 128, "padded"),        # two row tiles, the second partly filled
    ([400], 70, 9, 8, 128, 128, "hnd"),              # several row blocks
    ([333, 40], 35, 20, 8, 256, 64, "nhd"),
    ([900], 129, 2, 16, 32, 40, "hnd"),              # a draft longer than a tile, many row blocks
    ([1300, 128, 5], 5, 13, 8, 40, 120, "hnd"),
])
def test_tree_wide(lens, T, hk, G, page, D, layout, dt):
    assert scratch_of(lens, T, hk, G, page, D) > 0
    run_tree(dt, layout, lens, T, hk, G, page, D)


@pytest.mark.parametrize("T,hk,G", [(6, 40, 8), (48, 16, 8)])
def test_tree_wide_mask_kinds(T, hk, G):
    rng = np.random.default_rng(1)
    lens = [160, T, 300]
    assert scratch_of(lens, T, hk, G, 16, 64) > 0
    run_tree("f16", "hnd", lens, T, hk, G, 16, 64, mask=None)
    nothing = np.zeros((3, T, (T + 31) // 32), np.int32)
    got = run_tree("bf16", "hnd", lens, T, hk, G, 16, 64, mask=nothing)
    assert (host(got[1])[1] == -np.inf).all()
    dense = rng.integers(-2**31, 2**31, nothing.shape).astype(np.int32)
    run_tree("bf16", "nhd", lens, T, hk, G, 16, 64, mask=dense)
    run_tree("bf16", "hnd", [160, T, 300, 0, 9], T, hk, G, 16, 128, n_draft=[T, 3, 0, 0, 1])
    run_tree("bf16", "hnd", lens, T, hk, G, 16, 128, scale=30.0)
    run_tree("f16", "hnd", lens, T, hk, G, 16, 128, scale=1e-4)
    # a scale that is not positive goes another way
    run_tree("bf16", "hnd", lens, T, hk, G, 16, 128, scale=-0.2)
    run_tree("bf16", "hnd", lens, T, hk, G, 16, 128, scale=0.0)


@pytest.mark.parametrize("T,hk,G,D", [(6, 40, 8, 128), (48, 16, 8, 64)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_tree_wide_masked_infinities_and_nan(T, hk, G, D, dt):
    rng = np.random.default_rng(2)
    lens, page = np.array([290, 150], np.int32), 16
    assert scratch_of(lens, T, hk, G, page, D) > 0
    table, _ = tables(lens, page, 40, 20, rng)
    g = gen(3)
    k, v = (pool((40, hk, page, D), DTYPES[dt], "hnd", g) for _ in range(2))
    q = torch.randn((2, T, hk * G, D), device="cuda", generator=g).to(DTYPES[dt])
    sees = random_tree(rng, 2, T)
    sees[0, :, 1] = False
    sees[0, 1, 1] = sees[0, 3, 1] = True
    sees[0, :, 2] = False
    sees[0, 2, 2] = True
    clean = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens), mask=dev(mask_words(sees)))
    at = lambda p: (int(table[0, p // page]), slice(None), p % page)  # noqa: E731
    ctx = 290 - T
    x = v[at(ctx + 1)]
    x[:, : D // 2] = float("inf")
    x[:, D // 2] = float("nan")
    k[at(ctx + 2)] = float("nan")
    out, _ = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens), mask=dev(mask_words(sees)))
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[1, 3, 2]] = False
    assert torch.equal(out[0, keep], clean[0][0, keep]) and torch.equal(out[1], clean[0][1])
    for t in (1, 3):
        assert (out[0, t, :, : D // 2] == float("inf")).all() and out[0, t, :, D // 2].isnan().all()
        assert torch.equal(out[0, t, :, D // 2 + 1 :], clean[0][0, t, :, D // 2 + 1 :])
    assert out[0, 2].isnan().all()


def test_tree_wide_bad_pages_and_lengths():
    rng = np.random.default_rng(8)
    lens, T, hk, G = np.array([200, 150], np.int32), 12, 20, 8
    assert scratch_of(lens, T, hk, G, 16, 64) > 0
    table, _ = tables(lens, 16, 30, 14, rng)
    table[0, 3], table[0, 5], table[1, 9] = 30, -7, 1 << 30
    g = gen(4)
    k, v = (pool((30, hk, 16, 64), torch.bfloat16, "hnd", g) for _ in range(2))
    q = torch.randn((2, T, hk * G, 64), device="cuda", generator=g).bfloat16()
    got = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens))
    check_attention(*got, *kv_ref.tree_attention(host(q), host(k), host(v), table, lens), "bf16")
    err(ibp.IBP_ERANGE)
    lens = np.array([T - 1, 0], np.int32)  # drafts longer than their sequences
    got = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens))
    check_attention(*got, *kv_ref.tree_attention(host(q), host(k), host(v), table, lens), "bf16")
    err(ibp.IBP_ERANGE)


def test_tree_wide_strides_streams_graphs_and_the_same_bits():
    g = gen(6)
    lens, T, hk, G = np.array([900, 350, 60], np.int32), 9, 16, 8
    assert scratch_of(lens, T, hk, G, 16, 64) > 0
    table, _ = tables(lens, 16, 100, 60, np.random.default_rng(0))
    k, v = (pool((100, hk, 16, 64), torch.float16, "hnd", g) for _ in range(2))
    wide = torch.randn((3, T, 3, hk * G, 66), device="cuda", generator=g).half()
    q = wide[:, :, 1, :, :64]  # 4-byte aligned rows of a fused projection
    t, n = dev(table), dev(lens)
    want = kv.ibp_tree_attention(q.contiguous(), k, v, t, n)
    check_attention(*want, *kv_ref.tree_attention(host(q), host(k), host(v), table, lens), "f16")
    for _ in range(3):
        got = kv.ibp_tree_attention(q, k, v, t, n)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = kv.ibp_tree_attention(q, k, v, t, n, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kv.ibp_tree_attention(q, k, v, t, n)
        again = kv.ibp_tree_attention(q, k, v, t, n)
    for _ in range(20):
        graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(again[0], want[0])


def test_tree_wide_pool_past_32_bits():
    n, page, D, T, G = 70000, 256, 128, 128, 8
    assert scratch_of([600], T, 1, G, page, D) > 0
    k = torch.zeros((n, 1, page, D), dtype=torch.bfloat16, device="cuda")
    table = np.array([[n - 1, 3, n - 2]], np.int32)
    g = gen(1)
    for p in (n - 1, 3, n - 2):
        k[p].normal_(generator=g)
    q = torch.randn((1, T, G, D), device="cuda", generator=g).bfloat16()
    got = kv.ibp_tree_attention(q, k, k, dev(table), dev(np.array([600])))
    small, at = k[[n - 1, 3, n - 2]], np.array([[0, 1, 2]], np.int32)
    check_attention(*got, *kv_ref.tree_attention(host(q), host(small), host(small), at, np.array([600])), "bf16")


@pytest.mark.parametrize("T,G", [(2, 4), (16, 8), (40, 8)])
def test_tree_wide_long_ragged(T, G):
    """Ranges of many tiles that begin and end inside items, against the few-row kernel
    (every sequence by itself, a kv head at a time)."""
    lens = [9000, T, 4097, 300, 7001, 128, 2600]
    hk, page, D = 8, 64, 128
    assert scratch_of(lens, T, hk, G, page, D) > 0
    rng = np.random.default_rng(4)
    table, _ = tables(lens, page, 400, 142, rng)
    g = gen(9)
    k, v = (pool((400, hk, page, D), torch.bfloat16, "hnd", g) for _ in range(2))
    q = torch.randn((len(lens), T, hk * G, D), device="cuda", generator=g).bfloat16()
    words = dev(mask_words(random_tree(rng, len(lens), T)))
    t, n = dev(table), dev(np.array(lens))
    out, lse = kv.ibp_tree_attention(q, k, v, t, n, mask=words)
    for _ in range(30):
        again = kv.ibp_tree_attention(q, k, v, t, n, mask=words)
    assert torch.equal(again[0], out)
    for b in range(len(lens)):
        for h in (0, hk - 1):
            at = slice(h * G, h * G + G)
            keys = k[t[b].long().clamp(min=0), h].reshape(-1, D)[: lens[b]].double()
            vals = v[t[b].long().clamp(min=0), h].reshape(-1, D)[: lens[b]].double()
            bits = (words[b].long()[:, torch.arange(T, device="cuda") // 32] >> (torch.arange(T, device="cuda") % 32)) & 1
            sees = torch.cat([torch.ones(T, lens[b] - T, device="cuda"), bits], 1).bool()
            s = torch.einsum("tgd,nd->tgn", q[b, :, at].double(), keys) / math.sqrt(D)
            top = torch.einsum("tgd,nd->tgn", q[b, :, at].double().abs(), keys.abs()).amax(-1) / math.sqrt(D)
            s = s.masked_fill(~sees[:, None], -math.inf)
            p = torch.softmax(s, -1)
            want = [x.cpu().numpy() for x in (p @ vals, torch.logsumexp(s, -1), p @ vals.abs(), top)]
            check_attention(out[b, :, at], lse[b, :, at], *want, "bf16")


# ---------------------------------------------------------------------------
# Bounds and sparse attention


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lens,heads,page,D", [
    ([1], 1, 16, 64), ([100, 0, 64, 65], 3, 16, 128), ([50, 7], 2, 7, 40), ([400], 1, 128, 8), ([90, 31], 2, 1, 256),
    ([333, 200], 2, 24, 136),
])
def test_summarize(lens, heads, page, D, layout, dt):
    rng = np.random.default_rng(D)
    lens = np.array(lens, np.int32)
    n_pages = int((-(-lens // page)).sum()) + 2
    table, _ = tables(lens, page, n_pages, -(-int(lens.max()) // page) + 1, rng)
    k = pool((n_pages, heads, page, D), DTYPES[dt], layout, gen(D))
    poison(k, table, lens)
    k[table[0, 0], 0] *= 0  # a page of zeros
    if lens[0] > 1:
        k[table[0, (lens[0] - 1) // page], heads - 1, (lens[0] - 1) % page, D - 1] = float("-inf")
    for first in (None, np.maximum(lens - 20, 0).astype(np.int32), lens):
        codes = torch.full((n_pages, heads, 2, D), 55, dtype=torch.int8, device="cuda")
        scales = torch.full((n_pages, heads), 5.0, device="cuda")
        want = kv_ref.summarize(host(k), table, lens, host(codes), host(scales), first)
        kv.ibp_kv_summarize(k, dev(table), dev(lens), codes, scales, first=None if first is None else dev(first))
        assert np.array_equal(host(codes), want[0])
        assert np.array_equal(host(scales), want[1])


def run_sparse(dt, layout, lens, T, hk, G, page, D, budget, first, last, n_query=None, seed=0, coarse=False):
    rng = np.random.default_rng(seed)
    lens = np.array(lens, np.int32)
    B, n_pages = len(lens), int((-(-lens // page)).sum()) + 3
    table, _ = tables(lens, page, n_pages, max(1, -(-int(max(lens)) // page)) + 1, rng)
    g = gen(seed)
    k = pool((n_pages, hk, page, D), DTYPES[dt], layout, g)
    v = pool((n_pages, hk, page, D), DTYPES[dt], layout, g)
    if coarse:  # few different values: equal scores abound
        k.copy_(k.sign().nan_to_num())
    poison(k, table, lens)
    poison(v, table, lens)
    q = torch.randn((B, T, hk * G, D), device="cuda", generator=g).to(DTYPES[dt])
    if coarse:
        q = q.sign()
    codes = torch.zeros((n_pages, hk, 2, D), dtype=torch.int8, device="cuda")
    scales = torch.zeros((n_pages, hk), device="cuda")
    kv.ibp_kv_summarize(k, dev(table), dev(lens), codes, scales)
    out, lse, pages = kv.ibp_sparse_attention(q, k, v, dev(table), dev(lens), codes, scales, budget, keep_first=first,
                                              keep_last=last, n_query=None if n_query is None else dev(np.array(n_query)))
    want = kv_ref.sparse_attention(host(q), host(k), host(v), table, lens, host(codes), host(scales), budget, first,
                                   last, n_query)
    assert np.array_equal(host(pages), want[2])
    check_attention(out, lse, want[0], want[1], want[3], want[4], dt)
    return out, lse, pages


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lens,T,hk,G,page,D,budget,first,last", [
    ([1], 1, 1, 1, 16, 64, 1, 0, 1),
    ([600, 16, 17, 1], 1, 2, 4, 16, 128, 5, 1, 2),
    ([300, 90], 7, 2, 7, 24, 80, 4, 0, 1),
    ([200, 47], 9, 1, 16, 7, 40, 6, 2, 2),
    ([150], 3, 1, 20, 32, 128, 3, 1, 1),
    ([90, 65], 2, 2, 3, 64, 256, 2, 1, 1),
    ([300], 4, 1, 2, 1, 8, 40, 3, 30),
    ([130, 20], 11, 2, 1, 16, 136, 64, 0, 1),
])
def test_sparse_attention(lens, T, hk, G, page, D, budget, first, last, layout, dt):
    run_sparse(dt, layout, lens, T, hk, G, page, D, budget, first, last)


def test_sparse_equal_scores_take_the_lower_page():
    run_sparse("bf16", "hnd", [800, 500], 3, 2, 2, 4, 8, 40, 1, 1, coarse=True)


def test_sparse_long_and_large_budgets():
    run_sparse("bf16", "hnd", [9000], 1, 1, 4, 1, 64, 300, 1, 4)       # scores beyond shared memory
    run_sparse("f16", "hnd", [4000, 3000], 2, 1, 8, 16, 128, 100, 1, 2)


def test_sparse_ragged_queries():
    run_sparse("bf16", "hnd", [200, 100, 40, 0], 5, 2, 2, 16, 64, 3, 1, 1, n_query=[5, 2, 0, 0])


def test_sparse_of_every_page_is_tree_attention():
    g = gen(7)
    lens = np.array([500, 130], np.int32)
    table, _ = tables(lens, 16, 60, 40, np.random.default_rng(0))
    k, v = (pool((60, 2, 16, 64), torch.float16, "hnd", g) for _ in range(2))
    q = torch.randn((2, 3, 8, 64), device="cuda", generator=g).half()
    codes = torch.zeros((60, 2, 2, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((60, 2), device="cuda")
    kv.ibp_kv_summarize(k, dev(table), dev(lens), codes, scales)
    a = kv.ibp_sparse_attention(q, k, v, dev(table), dev(lens), codes, scales, 64)
    b = kv.ibp_tree_attention(q, k, v, dev(table), dev(lens))
    assert torch.allclose(a[0].float(), b[0].float(), atol=2e-3) and torch.allclose(a[1], b[1], atol=1e-5)


def test_sparse_infinite_queries_and_keys():
    """A key that is not finite marks its page; a query that is not finite scores nothing."""
    g = gen(7)
    lens = np.array([320], np.int32)
    table, _ = tables(lens, 16, 20, 20, np.random.default_rng(0))
    k, v = (pool((20, 1, 16, 64), torch.bfloat16, "hnd", g) for _ in range(2))
    k[table[0, 7], 0, 3, 5] = float("nan")
    q = torch.randn((1, 1, 2, 64), device="cuda", generator=g).bfloat16()
    codes = torch.zeros((20, 1, 2, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((20, 1), device="cuda")
    kv.ibp_kv_summarize(k, dev(table), dev(lens), codes, scales)
    out, _, pages = kv.ibp_sparse_attention(q, k, v, dev(table), dev(lens), codes, scales, 3, 0, 1)
    assert 7 in host(pages)[0, 0, 0].tolist() and out.isnan().all()
    q[0, 0, 1, 3] = float("inf")
    scales.nan_to_num_(posinf=0.0)
    _, _, pages = kv.ibp_sparse_attention(q, k, v, dev(table), dev(lens), codes, scales, 3, 0, 1)
    assert host(pages)[0, 0, 0].tolist() == [0, 1, 19]


# ---------------------------------------------------------------------------
# Random shapes, and refusals


def test_random_shapes():
    rng = random.Random(11)
    for i in range(40):
        page, D = rng.choice([1, 3, 8, 16, 24, 48, 64, 128, 160]), rng.choice([8, 24, 64, 72, 96, 128, 200, 256])
        hk, G, T = rng.choice([1, 2, 3]), rng.choice([1, 2, 5, 8]), rng.choice([1, 1, 2, 9, 31, 40])
        lens = [T + int(2 ** rng.uniform(0, 8.5)) for _ in range(rng.choice([1, 2, 4]))]
        dt, layout = rng.choice(["bf16", "f16"]), rng.choice(LAYOUTS)
        run_tree(dt, layout, lens, T, hk, G, page, D, seed=i)
        first, last = rng.choice([0, 1, 2]), rng.choice([1, 2])
        run_sparse(dt, layout, lens, min(T, 4), hk, G, page, D, first + last + rng.randrange(6), first, last, seed=i)


def test_refusals():
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    table, lens = dev(np.zeros((1, 2))), dev(np.array([20]))
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((4, 2, 2, 64), dtype=torch.int8, device="cuda")
    scales = torch.zeros((4, 2), device="cuda")
    tree = lambda **a: kv.ibp_tree_attention(**{**dict(q=q, k=k, v=k, table=table, lens=lens), **a})  # noqa: E731
    sparse = lambda **a: kv.ibp_sparse_attention(**{**dict(q=q, k=k, v=k, table=table, lens=lens, codes=codes,  # noqa: E731
                                                          scales=scales, budget=2), **a})
    tree(), sparse()
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(table=table.long()), dict(lens=dev(np.array([1, 2]))),
                dict(q=q[..., :32]), dict(mask=dev(np.zeros((1, 1, 2)))), dict(n_draft=dev(np.array([1, 1]))),
                dict(out=torch.empty_like(q)[..., :32]), dict(v=k.half()), dict(k=k.cpu()), dict(k=k[0]),
                # enough work to need scratch
                dict(table=dev(np.zeros((64, 60))), lens=dev(np.full(64, 20)), q=q.expand(64, 1, 4, 64),
                     workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(ValueError):
            tree(**bad)
    for bad in (dict(budget=0), dict(budget=5000), dict(keep_last=0), dict(keep_first=2), dict(codes=codes[:3]),
                dict(scales=scales.double()), dict(n_query=dev(np.array([1, 1])))):
        with pytest.raises(ValueError):
            sparse(**bad)
    odd = torch.zeros((4, 2, 16, 68), dtype=torch.bfloat16, device="cuda")
    q5 = torch.zeros((1, 1, 5, 64), dtype=torch.bfloat16, device="cuda")
    big = torch.zeros((4, 1, 1, 264), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(k=odd[..., :64], v=odd[..., :64]), dict(q=q5), dict(scale=math.nan),
                dict(k=big, v=big, q=torch.zeros((1, 1, 1, 264), dtype=torch.bfloat16, device="cuda")),
                dict(v=k[:3])):
        with pytest.raises(ibp.IbpError, match="IBP_EINVAL.*\\("):
            tree(**bad)
    refs, rows = dev(np.zeros(4)), dev(np.array([0]))
    with pytest.raises(ibp.IbpError, match="page_tokens"):
        kv.ibp_kv_fork(table, lens, refs, rows, 0)
    with pytest.raises(ValueError):
        kv.ibp_kv_copy(k, dev(np.zeros((1, 2))), rows)
    with pytest.raises(ValueError):
        kv.ibp_kv_accept(k, table, lens, dev(np.zeros(3)), rows, dev(np.zeros((1, 1))), rows)
    with pytest.raises(ValueError):
        kv.ibp_kv_summarize(k, table, lens, codes.int(), scales)
    lib = kv._load()
    seqs = kv._Seqs(table.data_ptr(), lens.data_ptr(), 1, 2)
    # overlapping tables, a scratch that is too small, pageable memory
    one = torch.zeros(8, dtype=torch.int32, device="cuda")
    args = lambda t, size: (seqs, 16, refs.data_ptr(), 4, rows.data_ptr(), 1, t, one.data_ptr(), refs.data_ptr(),  # noqa: E731
                            one.data_ptr(), one.data_ptr(), one.data_ptr(), size, None, None)
    assert lib.ibp_kv_fork(*args(table.data_ptr(), 1 << 20)) == ibp.IBP_EINVAL
    assert b"overlap" in lib.ibp_last_error_detail()
    assert lib.ibp_kv_fork(*args(one.data_ptr(), 8)) == ibp.IBP_EINVAL
    page = ctypes.create_string_buffer(64)
    assert lib.ibp_kv_fork(*args(ctypes.addressof(page), 1 << 20)) == ibp.IBP_EINVAL
    assert lib.ibp_tree_attention(None, None, 0, seqs, None, 0, 0, 0, 1, 1, None, None, 1.0, None, None, None, 0, None,
                                  None) == ibp.IBP_EINVAL


def test_own_status_word():
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv.ibp_kv_free(dev(np.array([[0]])), dev(np.array([1])), dev(np.array([1])), dev(np.array([4])), 16, status=word)
    assert word.item() == ibp.IBP_ERANGE
    with pytest.raises(ibp.IbpError, match="IBP_ERANGE"):
        kv.ibp_kv_free(dev(np.array([[0]])), dev(np.array([1])), dev(np.array([1])), dev(np.array([4])), 16)
        kv.ibp_kv_get_status()


def test_no_sequences():
    none = torch.empty((0, 3), dtype=torch.int32, device="cuda")
    lens = torch.empty(0, dtype=torch.int32, device="cuda")
    k = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((0, 2, 4, 64), dtype=torch.bfloat16, device="cuda")
    assert kv.ibp_tree_attention(q, k, k, none, lens)[0].shape == q.shape
    codes, scales = torch.zeros((4, 2, 2, 64), dtype=torch.int8, device="cuda"), torch.zeros((4, 2), device="cuda")
    assert kv.ibp_sparse_attention(q, k, k, none, lens, codes, scales, 4)[2].shape == (0, 2, 2, 4)
    kv.ibp_kv_summarize(k, none, lens, codes, scales)
    refs = dev(np.array([1, 0, 2, 0]))
    assert host(kv.ibp_kv_fork(none, lens, refs, lens, 16)[2]).tolist() == [1, 0, 2, 0]
    assert host(kv.ibp_kv_compact(none, refs, 16)[1]).tolist() == [1, 2, 0, 0]


def test_the_example_runs_the_operators_together():
    """examples/kv_serving.py: compressed host cache, pages, sparse step, beams, tree, acceptance, compaction."""
    import importlib.util
    import os

    at = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "kv_serving.py")
    spec = importlib.util.spec_from_file_location("kv_serving", at)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    from host_transfer_gb300 import workloads

    seq, heads, page = 260, 2, 32
    r = example.run(seq=seq, heads=heads, group=4, page=page, beams=3, budget=4)
    a, b = r["first"], r["second"]
    # the pages hold the prompt's keys bit for bit
    for s, n in enumerate(host(a["lens"])):
        words = workloads.llm_kv(s, heads=heads, seq=seq, head_dim=128)
        for pages, w in zip((a["k"], a["v"]), words):
            bits = pages.view(torch.int16).cpu().numpy().view(np.uint32)
            for h in range(heads):
                got = np.concatenate([bits[p, h] for p in host(a["table"])[s][: -(-n // page)]])[:n]
                assert np.array_equal(got, w.reshape(heads, seq, 64)[h, :n])
    want = kv_ref.sparse_attention(host(a["q"]), host(a["k"]), host(a["v"]), host(a["table"]), host(a["lens"]),
                                   host(a["codes"]), host(a["scales"]), a["budget"], 1, 2)
    assert np.array_equal(host(a["pages"]), want[2])
    check_attention(a["out"], a["lse"], want[0], want[1], want[3], want[4], "bf16")
    check_attention(b["out"], b["lse"], *kv_ref.tree_attention(host(b["q"]), host(b["k"]), host(b["v"]), host(b["table"]),
                                                               host(b["lens"]), host(b["mask"])), "bf16")
    # compaction moved pages, not what sequences hold
    refs, table, lens = host(r["refs"]), host(r["table"]), host(r["lens"])
    assert r["moved"] > 0 and (refs[: (refs > 0).sum()] > 0).all()
    for s, n in enumerate(lens):
        for p in range(-(-n // page)):
            assert torch.equal(r["pool"][:, table[s, p]], r["before"]["pool"][:, int(r["before"]["table"][s, p])])
