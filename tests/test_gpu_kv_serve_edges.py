"""GPU tests of the calls around the caches in 4 bits, verification and eviction that
hand one's results to the next, and of their less usual layouts, against the CPU oracle."""

import numpy as np
import pytest
import torch

from host_transfer_gb300 import ibp, kv
from oracle import kv_ref, kv_serve_ref as ref
from tests.kv_util import DTYPES, check_attention, dev, host, pool, tables
from tests.test_gpu_kv_serve import Cache, check_weigh, gen, unheld

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


def forked(lens, page, seed=0, extra=2):
    """Sequences, and a fork of each: (table, lens, refs) with the full pages shared."""
    rng = np.random.default_rng(seed)
    n = len(lens)
    lens = np.array(lens, np.int32)
    width = -(-int(lens.max()) // page) + 1
    table, refs = tables(lens, page, int((-(-lens // page)).sum()) + n + extra, width, rng)
    pages = torch.randn((len(refs), 2, page, 16), device="cuda", generator=gen(seed)).bfloat16()
    got = kv.ibp_kv_fork(dev(table), dev(lens), dev(refs), dev(np.repeat(np.arange(n), 2)), page)
    kv.ibp_kv_copy(pages, *got[3:])
    return pages, *got[:3]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("evicted", [(0,), (0, 1), (1, 2, 3)])
def test_evicting_a_fork_leaves_its_sibling_alone(evicted, inplace):
    """Moving a fork's tokens to the front would overwrite pages that another sequence holds:
    a sequence of whose targets one is shared stays as it is, and the status says so."""
    page, budget = 16, 40
    pages, table, lens, refs = forked([100, 64], page, extra=4)
    # a sequence of its own beside them, which moves
    own = np.flatnonzero(host(refs) == 0)[:4].astype(np.int32)
    assert len(own) == 4 or pytest.fail("no pages left")
    row = np.full((1, table.shape[1]), -1, np.int32)
    row[0, :4] = own
    table, lens = torch.cat([table, dev(row)]), torch.cat([lens, dev(np.array([60]))])
    refs[torch.from_numpy(own).cuda().long()] = 1
    rng = np.random.default_rng(5)
    w = rng.random((5, 112)).astype(np.float32)
    path, n_draft, n_keep, _ = kv.ibp_kv_evict(dev(w, torch.float32), lens, budget, keep_first=2, keep_last=3)
    others = [b for b in range(4) if b not in evicted]
    n_draft[others] = 0
    n_keep[others] = 0
    before = host(pages).copy()
    want = kv_ref.accept(before, *map(host, (table, lens, refs, n_draft, path, n_keep)))
    got = kv.ibp_kv_accept(pages, table, lens, refs, n_draft, path, n_keep, inplace=inplace)
    err(ibp.IBP_EINVAL)
    assert np.array_equal(host(pages), want[0])
    assert all(np.array_equal(host(x), y) for x, y in zip(got, want[1:]))
    assert host(got[1]).tolist() == [100, 100, 64, 64, budget]
    changed = (want[0] != before).any((1, 2, 3))
    assert set(np.flatnonzero(changed)) <= set(own.tolist()) and changed.any()


@pytest.mark.parametrize("inplace", [False, True])
def test_sharing_is_judged_before_any_page_is_freed(inplace):
    """One row gives a shared page up while another wants to write it: both in one call."""
    page = 8
    # rows 0 and 1 share pages 0 and 1; row 2 is on its own
    table, lens = np.array([[0, 1, -1], [0, 1, 2], [3, 4, -1]], np.int32), np.array([16, 20, 16], np.int32)
    refs = np.array([2, 2, 1, 1, 1, 0], np.int32)
    n_draft, n_keep = np.array([16, 20, 16], np.int32), np.array([3, 12, 10], np.int32)
    path = np.full((3, 12), -1, np.int32)
    path[0, :3] = [0, 1, 2]  # nothing moves, page 1 is given up
    path[1] = np.arange(8, 20)  # writes pages 0 and 1
    path[2, :10] = np.arange(6, 16)
    pages = torch.arange(6 * page * 4, device="cuda", dtype=torch.float32).reshape(6, 1, page, 4)
    want = kv_ref.accept(host(pages), table, lens, refs, n_draft, path, n_keep)
    got = kv.ibp_kv_accept(pages, *map(dev, (table, lens, refs, n_draft, path, n_keep)), inplace=inplace)
    err(ibp.IBP_EINVAL)
    assert np.array_equal(host(pages), want[0])
    assert all(np.array_equal(host(x), y) for x, y in zip(got, want[1:]))
    assert host(got[1]).tolist() == [3, 20, 10] and host(got[2]).tolist() == [2, 1, 1, 1, 1, 0]


def test_a_draft_behind_a_shared_prefix_is_accepted():
    """Only the pages that are written have to be a sequence's own."""
    page, T = 16, 9
    rng = np.random.default_rng(3)
    pages, table, lens, refs = forked([77, 64, 40], page, seed=3, extra=12)
    free = iter(np.flatnonzero(host(refs) == 0))
    t, r, n = host(table).copy(), host(refs).copy(), host(lens) + T
    for b in range(6):
        for p in range(-(-int(n[b] - T) // page), -(-int(n[b]) // page)):
            t[b, p] = next(free)
            r[t[b, p]] = 1
    n_draft, n_accept = np.full(6, T, np.int32), np.array([3, 9, 0, 5, 4, 1], np.int32)
    path = np.full((6, T), -1, np.int32)
    for b in range(6):
        path[b, : n_accept[b]] = np.sort(rng.permutation(T)[: n_accept[b]])
    assert (r > 1).any()
    want = kv_ref.accept(host(pages), t, n, r, n_draft, path, n_accept)
    got = kv.ibp_kv_accept(pages, *map(dev, (t, n, r, n_draft, path, n_accept)))
    assert np.array_equal(host(pages), want[0]) and host(got[1]).tolist() == (n - T + n_accept).tolist()
    assert all(np.array_equal(host(x), y) for x, y in zip(got, want[1:]))


@pytest.mark.parametrize("page", [16, 24])
def test_a_long_eviction_and_its_move(page):
    """A budget of 8192 tokens over several sequences, codes and scales, the lengths and references once."""
    lens, budget, dim = [20000, 8192, 12345, 9000], 8192, 64
    c = Cache(lens, 1, 2, 1, page, dim, seed=9)
    rng = np.random.default_rng(9)
    w = rng.random((4, 20480)).astype(np.float32)
    path, n_draft, n_keep, left = kv.ibp_kv_evict(dev(w, torch.float32), c.lens, budget, keep_first=4, keep_last=1024)
    want = ref.evict(w, lens, budget, 4, 1024)
    assert all(np.array_equal(host(x), y) for x, y in zip((path, n_draft, n_keep, left), want))
    for x in (*c.k, *c.v):
        bits = x.view(torch.int16) if x.dtype != torch.uint8 else x  # NaN where no token is
        moved = kv_ref.accept(host(bits), c.np_table, c.np_lens, c.np_refs, want[1], want[0], want[2])
        got = kv.ibp_kv_accept(x, c.table, c.lens, c.refs, n_draft, path, n_keep)
        assert np.array_equal(host(bits), moved[0])
        assert all(np.array_equal(host(a), b) for a, b in zip(got, moved[1:]))


# ---------------------------------------------------------------------------
# Layouts


def loose(q):
    """The same queries with a base and strides that are multiples of 4 bytes only."""
    B, T, H, D = q.shape
    wide = torch.full((B, T, H, D + 6), float("nan"), dtype=q.dtype, device="cuda")
    wide[..., 2 : D + 2] = q
    return wide[..., 2 : D + 2]


@pytest.mark.parametrize("layout,strided", [("hnd", True), ("nhd", False), ("padded", True), ("padded", False)])
@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D", [
    ([70, 0, 33], 1, 2, 4, 16, 64), ([300, 17], 1, 8, 1, 7, 128), ([60, 90], 2, 3, 2, 24, 256),  # 8 rows at most
    ([100, 64, 80], 5, 3, 2, 24, 96), ([90, 41], 20, 2, 2, 16, 128), ([50, 41], 30, 1, 3, 64, 256),  # few rows
    ([300, 90], 70, 3, 1, 16, 64), ([700], 40, 1, 8, 24, 128), ([300, 120], 17, 4, 5, 7, 96),  # tensor cores
])
def test_weigh_in_every_layout(lens, T, hk, G, page, D, dt, four, layout, strided):
    c = Cache(lens, T, hk, G, page, D, dt, layout, seed=D + T)
    n_draft = np.array([max(0, min(T - i, n)) for i, n in enumerate(lens)], np.int32)
    keys = c.k
    if not four:
        keys = pool(c.np_k.shape, DTYPES[dt], layout, gen(1), fill=float("nan"))
        keys.copy_(torch.from_numpy(c.np_k).to("cuda"))
        keys.masked_fill_(unheld(c.np_table, c.np_lens, keys.shape[0], page), float("nan"))
    lse = c.want(n_draft)[1].astype(np.float32)
    width = c.np_table.shape[1] * page + 3
    was = np.random.default_rng(1).random((len(lens), width)).astype(np.float32)
    want, top = ref.weigh(host(c.q), c.np_k, c.np_table, c.np_lens, lse, was, None, n_draft, decay=0.75)
    got = kv.ibp_kv_weigh(loose(c.q) if strided else c.q, keys, c.table, c.lens, dev(lse, torch.float32), dev(was, torch.float32),
                          n_draft=dev(n_draft), decay=0.75)
    check_weigh(got, want, top, lse, T * hk * G, was, 0.75)


MANY = [  # (sequences, drafted tokens, kv heads, heads of each, page, dim): tensor cores on codes
    ([300, 290] * 3, 17, 2, 8, 64, 128), ([200, 141, 150] * 3, 100, 3, 1, 7, 64), ([170] * 12, 130, 2, 1, 16, 96),
    ([310, 305, 301], 100, 2, 5, 24, 128),
    # more than 512 rows: decoded once
    ([310, 305, 301], 130, 2, 4, 16, 128), ([600, 641], 600, 1, 1, 7, 64), ([310, 303], 260, 2, 3, 24, 96),
]


@pytest.mark.parametrize("layout,strided", [("hnd", True), ("nhd", False), ("padded", True), ("padded", False)])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D", MANY)
def test_attention_of_many_rows_in_every_layout(lens, T, hk, G, page, D, dt, layout, strided):
    """Scratch begins as NaN: what a call does not write there must not matter."""
    c = Cache(lens, T, hk, G, page, D, dt, layout, seed=T, mask=True)
    assert -(-max(lens) // 128) * len(lens) * hk * -(-T * G // 16) >= 304, "work enough for the tensor cores"
    live = np.array([T - (i % 3) for i in range(len(lens))], np.int32)
    size = kv._load().ibp_kv4_attention_workspace(len(lens), c.np_table.shape[1], page, T, hk * G, hk, D)
    want = c.want(live)
    if strided:
        c.q = loose(c.q)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    check_attention(*c.attend(n_draft=dev(live), workspace=ws), *want, dt)


@pytest.mark.parametrize("layout", ["hnd", "padded"])
@pytest.mark.parametrize("T,hk,G,D", [(260, 2, 3, 128), (100, 1, 12, 64)])
def test_many_rows_over_a_table_too_wide_to_decode(T, hk, G, D, layout):
    """Scratch goes by the table's width; where the decoded cache would pass 4 GB there, calls
    of more than 512 rows read codes too."""
    c = Cache([700, T, 500], T, hk, G, 64, D, "bf16", layout, seed=T, mask=True)
    live = np.array([T, T - 1, T - 2], np.int32)
    want = c.want(live)
    wide = torch.full((3, 120000), -1, dtype=torch.int32, device="cuda")
    wide[:, : c.table.shape[1]] = c.table
    size = kv._load().ibp_kv4_attention_workspace(3, 120000, 64, T, hk * G, hk, D)
    assert size < 1 << 30 < 3 * 120000 * 64 * hk * D * 4 // 4
    c.table = wide
    check_attention(*c.attend(n_draft=dev(live), workspace=torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")), *want, "bf16")


# ---------------------------------------------------------------------------
# Values past the type's range


@pytest.mark.parametrize("T,hk,G,page", [(3, 1, 2, 16), (7, 2, 1, 24), (13, 1, 4, 16), (70, 8, 4, 16)])
def test_half_precision_values_past_its_range_are_infinite(T, hk, G, page):
    """Scale 9000 stands for 0 (code 8) and -infinity (code 0: -72000): a row that sees such a
    value has the infinity there and its ordinary output beside it."""
    lens = [T + 30, T + 900, T]
    c = Cache(lens, T, hk, G, page, 64, "f16", seed=T)
    odd = T - 2
    sees = np.random.default_rng(7).random((3, T, T)) < 0.5
    sees[:, :, odd] = np.arange(T) % 2 == 1
    bits = np.zeros((3, T, -(-T // 32)), np.uint32)
    for t in range(T):
        for i in range(T):
            bits[:, t, i // 32] |= (sees[:, t, i].astype(np.uint32) << np.uint32(i % 32)).astype(np.uint32)
    c.np_mask, c.mask = bits, dev(bits.view(np.int32))
    for b in range(3):
        pos = lens[b] - T + odd
        at = int(c.np_table[b, pos // page]), hk - 1, pos % page
        c.v[0][at], c.v[1][at] = 0x08, 9000.0
        c.np_v[at] = 0.0  # what the even elements stand for
    out, lse = c.attend()
    want, want_lse, mean, top = c.want()
    seen = torch.from_numpy(sees[:, :, odd]).cuda()
    last = out[:, :, (hk - 1) * G :]
    assert (last[seen][..., 1::2] == -float("inf")).all()
    got = out.clone()
    got[:, :, (hk - 1) * G :][..., 1::2][seen] = torch.from_numpy(want).cuda()[:, :, (hk - 1) * G :][..., 1::2][seen].half()
    check_attention(got, lse, want, want_lse, mean, top, "f16")


# ---------------------------------------------------------------------------
# Clusters


def test_calls_of_clusters_agree_with_the_oracle_every_time():
    """What one lane of a CTA writes before the cluster's barrier is there for all behind it."""
    rng = np.random.default_rng(11)
    B, width, budget, V, T = 12, 20001, 700, 20000, 5
    w = np.round(rng.random((B, width)) * 50).astype(np.float32)  # many equal weights: every count is used
    lens = rng.integers(budget, width + 1, B).astype(np.int32)
    evicted = ref.evict(w, lens, budget, 3, 90)
    p, q = (rng.random((B, T + i, V)).astype(np.float32) ** 6 for i in (1, 0))
    p, q = p / p.sum(-1, keepdims=True), q / q.sum(-1, keepdims=True)
    tokens = rng.integers(0, V, (B, T)).astype(np.int32)
    parents = np.maximum(np.arange(T) - rng.integers(1, 4, (B, T)), -1).astype(np.int32)
    u = rng.random((B, T + 1)).astype(np.float32)
    verified = ref.verify(p, tokens, u, q, parents)[:3]
    # 200 sequences: the bookkeeping of an acceptance is a cluster's
    page, draft = 8, 20
    n = rng.integers(draft, 60, 200).astype(np.int32)
    table, refs = tables(n, page, 2000, 8, rng)
    count = rng.integers(0, draft + 1, 200).astype(np.int32)
    path = np.stack([np.sort(rng.permutation(draft)) for _ in n]).astype(np.int32)
    for b, c in enumerate(count):
        path[b, :c] = np.sort(rng.permutation(draft)[:c])
    pages = torch.randn((2000, 2, page, 16), device="cuda", generator=gen(3)).bfloat16()
    accepted = kv_ref.accept(host(pages), table, n, refs, np.full(200, draft), path, count)
    args = dev(w, torch.float32), dev(lens)
    drafts = dev(p, torch.float32), dev(tokens), dev(u, torch.float32), dev(q, torch.float32), dev(parents)
    rows = [dev(x) for x in (table, n, refs, np.full(200, draft), path, count)]
    for _ in range(20):
        got = kv.ibp_kv_evict(*args, budget, keep_first=3, keep_last=90)
        assert all(np.array_equal(host(x), y) for x, y in zip(got, evicted))
        assert all(np.array_equal(host(x), y) for x, y in zip(kv.ibp_kv_verify(*drafts), verified))
        x = pages.clone()
        got = kv.ibp_kv_accept(x, *rows)
        assert np.array_equal(host(x), accepted[0]) and all(np.array_equal(host(x), y) for x, y in zip(got, accepted[1:]))
