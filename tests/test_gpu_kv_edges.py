"""GPU tests of the paged key/value cache operators where a call's data, values or
surroundings are out of the ordinary."""

import ctypes
import threading

import numpy as np
import pytest
import torch

from host_transfer_gb300 import ibp, kv
from oracle import kv_ref
from tests.kv_util import DTYPES, check_attention, dev, host, pool, tables

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def clean_status():
    yield
    assert kv.ibp_kv_get_status(raise_on_error=False) == ibp.IBP_OK


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def err(code):
    """The status the test has provoked, read and cleared."""
    assert kv.ibp_kv_get_status(raise_on_error=False) == code


class Cache:
    """A small cache with the bounds of its keys, and queries."""

    def __init__(self, lens, T, hk, G, page, D, dt="bf16", seed=0, spare=3):
        rng = np.random.default_rng(seed)
        self.np_lens = np.array(lens, np.int32)
        n_pages = int((-(-self.np_lens // page)).sum()) + spare
        self.np_table, self.np_refs = tables(lens, page, n_pages, max(1, -(-int(max(lens)) // page)) + 1, rng)
        g = gen(seed)
        self.k, self.v = (pool((n_pages, hk, page, D), DTYPES[dt], "hnd", g) for _ in range(2))
        self.q = torch.randn((len(lens), T, hk * G, D), device="cuda", generator=g).to(DTYPES[dt])
        self.table, self.lens, self.refs = dev(self.np_table), dev(self.np_lens), dev(self.np_refs)
        self.codes = torch.zeros((n_pages, hk, 2, D), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((n_pages, hk), device="cuda")
        kv.ibp_kv_summarize(self.k, self.table, self.lens, self.codes, self.scales)

    def sparse(self, budget, **kw):
        return kv.ibp_sparse_attention(self.q, self.k, self.v, self.table, self.lens, self.codes, self.scales, budget, **kw)

    def tree(self, **kw):
        return kv.ibp_tree_attention(self.q, self.k, self.v, self.table, self.lens, **kw)


# ---------------------------------------------------------------------------
# Counts of queries and drafted tokens above T


@pytest.mark.parametrize("page", [16, 7])  # whole steps a page, and steps that cross pages
@pytest.mark.parametrize("T,more", [(1, 1), (1, 1989), (3, 2), (9, 60), (2, 2**31 - 3)])
def test_more_queries_than_rows(T, more, page):
    """n_query above T is an error; the call gives what n_query = T gives."""
    c = Cache([2000, 40, 300], T, 2, 2, page, 64)
    want = c.sparse(8, keep_first=1, keep_last=2)
    got = c.sparse(8, keep_first=1, keep_last=2, n_query=dev(np.full(3, T + more)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    err(ibp.IBP_ERANGE)


@pytest.mark.parametrize("T,hk,G", [(3, 2, 2), (24, 16, 8)])
def test_more_drafted_tokens_than_rows(T, hk, G):
    c = Cache([700, 60, 300], T, hk, G, 16, 64)
    want = c.tree()
    got = c.tree(n_draft=dev(np.full(3, T + 5)))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    err(ibp.IBP_ERANGE)


# ---------------------------------------------------------------------------
# Values


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("form,page,D,G", [
    ("tree", 20, 64, 1), ("tree", 20, 136, 3),      # few rows
    ("tree", 64, 64, 4), ("tree", 64, 128, 136),    # tensor cores: one row tile, two
    ("sparse", 64, 64, 2), ("sparse", 20, 128, 2),
])
def test_a_long_tail_under_one_key(form, page, D, G, dt):
    """One key outweighs 65536 others of e^-17.55 (2^-25.3) each, which are 0.16 % of
    the output together and all of it where the one key's value is zero.  Sequences
    enough that no row is shared out over CTAs with maxima of their own."""
    n, B = 65537, 320
    c = Cache([n], 1, 1, G, page, D, dt)
    c.k.zero_(), c.q.zero_(), c.v.uniform_(0.5, 1.5, generator=gen(3))
    c.k[..., 0] = -17.546875 if dt == "f16" else -17.5
    c.q[..., 0] = 1
    first = int(c.np_table[0, 0]), 0, 0
    c.k[first] = 0
    c.v[first] = 0
    want = kv_ref.tree_attention(host(c.q), host(c.k), host(c.v), c.np_table, c.np_lens, scale=1.0)
    assert (want[0] > 1e-3).all()
    c.table, c.lens, c.q = c.table.repeat(B, 1), c.lens.repeat(B), c.q.repeat(B, 1, 1, 1)
    if form == "tree":
        out, lse = c.tree(scale=1.0)
    else:
        out, lse, _ = c.sparse(4096, scale=1.0)
    check_attention(out, lse, *(x.repeat(B, 0) for x in want), dt)


@pytest.mark.parametrize("G,page", [(2, 20), (4, 64), (136, 64)])
def test_scores_of_all_magnitudes_in_half_precision(G, page):
    """The powers stay within half precision where single precision is coarse: scores
    from 2^-10 to 2^34 in steps, of either sign, equal ones side by side."""
    D, n = 64, 300
    c = Cache([n] * 140, 1, 2, G, page, D, "f16")
    c.k.zero_(), c.q.zero_()
    c.k[..., 0] = 1
    c.q[..., 0] = 1
    c.v.fill_(1.5)
    for sign in (1, -1):
        for e in range(-10, 35):
            c.k[..., 0] = sign * 2.0 ** min(e, 15) * (1 + 2.0**-10)
            out, lse = c.tree(scale=2.0 ** max(0, e - 15))
            # every probability is rounded alike (2^-11), then the output is (2^-11); sums in 32 bits
            assert ((out.double() - 1.5).abs() <= 1.5 * (2 * 2.0**-11 + 2.0**-15)).all()
            score = sign * 2.0**e * (1 + 2.0**-10)
            assert torch.allclose(lse.double(), torch.full_like(lse, 1).double() * (score + np.log(n)), rtol=2.0**-21, atol=2.0**-19)


@pytest.mark.parametrize("dt,low", [("bf16", -3.3895313892515355e38), ("f16", -65504.0)])
@pytest.mark.parametrize("G,page", [(2, 20), (4, 64), (136, 64)])
def test_keys_of_the_lowest_value(G, page, dt, low):
    """A row whose keys all give the type's lowest value is a mean like any other, and
    beside ordinary keys they weigh nothing."""
    n, D = 300, 64
    c = Cache([n] * 140, 1, 2, G, page, D, dt)
    c.k.zero_(), c.q.zero_()
    c.k[..., 0] = low
    c.q[..., 0] = 1
    out, lse = c.tree()
    few = slice(0, 3)
    want = kv_ref.tree_attention(host(c.q)[few], host(c.k), host(c.v), c.np_table[few], c.np_lens[few])
    u = 2.0**-8 if dt == "bf16" else 2.0**-11  # equal probabilities: rounded once, then the output
    assert (np.abs(host(out)[few] - want[0]) <= (2 * u + 2.0**-15) * want[2] + 2.0**-25).all()
    assert torch.equal(out.isfinite(), torch.ones_like(out, dtype=torch.bool)) and lse.isfinite().all()
    c.k[:, :, 5::16, 0] = 0.25  # at least one in a tile of each row
    out, lse = c.tree()
    want = kv_ref.tree_attention(host(c.q)[few], host(c.k), host(c.v), c.np_table[few], c.np_lens[few])
    # the kept keys' scores are equal: the same bound
    assert (np.abs(host(out)[few] - want[0]) <= (2 * u + 2.0**-15) * want[2] + 2.0**-25).all()
    assert np.abs(host(lse)[few] - want[1]).max() <= 2.0**-19


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("n,T,G,page", [
    (6000, 16, 8, 16), (6000, 40, 8, 64),   # tensor cores, ranges of a few tiles
    (900, 3, 2, 16), (20000, 3, 2, 20),     # few rows: joined in a cluster, by a second kernel
])
def test_infinite_values_of_no_weight_are_seen_in_every_part(n, T, G, page, dt):
    """One key of the context outweighs all others by 2^-288, so the parts of a split
    row that hold the draft have weight 0; a drafted value that is not finite
    decides the rows that see it all the same."""
    D = 64
    c = Cache([n], T, 1, G, page, D, dt)
    c.k.zero_(), c.q.zero_()
    c.q[..., 0] = 1
    top = int(c.np_table[0, 0]), 0, 1
    c.k[top][0] = 200
    sees = np.tril(np.ones((T, T), bool))
    sees[0, 0] = False  # row 0 sees no drafted token; token 1 is the infinite one
    sees[T - 1, 1] = False
    words = np.zeros((1, T, (T + 31) // 32), np.uint32)
    for i in range(T):
        words[0, :, i // 32] |= sees[:, i].astype(np.uint32) << np.uint32(i % 32)
    mask = dev(words.view(np.int32))
    clean, lse = c.tree(mask=mask, scale=1.0)
    assert torch.equal(clean, c.v[top].expand_as(clean))
    at = n - T + 1
    c.v[int(c.np_table[0, at // page]), 0, at % page, 3] = float("inf")
    c.v[int(c.np_table[0, at // page]), 0, at % page, 7] = float("nan")
    out, lse2 = c.tree(mask=mask, scale=1.0)
    assert torch.equal(lse, lse2)
    hit = torch.from_numpy(sees[:, 1]).cuda()
    assert torch.equal(out[0, ~hit], clean[0, ~hit])
    assert not out[0, hit][..., [3, 7]].isfinite().any()
    keep = [d for d in range(D) if d not in (3, 7)]
    assert torch.equal(out[..., keep], clean[..., keep])


# ---------------------------------------------------------------------------
# Order on the stream


def test_early_fetch_behind_two_calls_reads_what_the_first_wrote():
    """Compressed rows move as pages, another call follows, then a decode with the
    early-fetch hint: the kernel just before it wrote none of its inputs, the one
    before that all of them."""
    n, W = 200000, 128
    g = gen(1)
    tables_ = [torch.randint(0, 1 << 20, (n, W), generator=g, device="cuda", dtype=torch.int32) | (5 << 24) for _ in range(2)]
    plan = ibp.ibp_plan_create(*ibp.ibp_preprocess(tables_[0][:4096].contiguous(), 0.99))
    old, new = [ibp.ibp_compress(plan, t.clone()) for t in tables_]
    assert torch.equal(old[1], new[1])  # every row of both is compressed
    pages = torch.empty((2 * n, 1, 1, W), dtype=torch.int32, device="cuda")
    pages[n:, 0, 0] = new[0]
    rows = torch.arange(n, dtype=torch.int32, device="cuda")
    moves = torch.stack([rows + n, rows, torch.ones_like(rows)], 1).contiguous()
    count, ids = dev(np.array([n])), torch.randperm(n, generator=g, device="cuda")
    small = dev(np.array([[0, -1]])), dev(np.array([5])), dev(np.array([1, 0])), dev(np.array([0]))
    plan.set_hints(ibp.IBP_HINT_EARLY_FETCH)
    for _ in range(10):
        pages[:n, 0, 0] = old[0]
        torch.cuda.synchronize()
        kv.ibp_kv_copy(pages, moves, count)
        kv.ibp_kv_free(*small, 16)
        out = ibp.ibp_gather_decompress(plan, pages[:n, 0, 0], new[1], ids)
        assert torch.equal(out, tables_[1][ids])
    assert ibp.ibp_get_status(plan) == ibp.IBP_OK


class Step:
    """A pass through every call but tree attention, on buffers of its own: a fork with its
    copies, bounds, sparse attention, an acceptance, a free, a compaction.  The lengths leave
    room for the draft in a row's last page, its own after the fork."""

    def __init__(self, seed, lens=(300, 77, 139), T=2, page=16, D=64, dt="bf16"):
        self.page, rng = page, np.random.default_rng(seed)
        table, refs = tables(list(lens), page, 70, -(-max(lens) // page) + 2, rng)
        g = gen(seed)
        self.first = dict(pool=torch.randn((2, 70, 2, page, D), device="cuda", generator=g).to(DTYPES[dt]), table=dev(table),
                          lens=dev(np.array(lens)), refs=dev(refs), parents=dev(rng.integers(0, 3, 4)),
                          n_draft=dev(np.full(4, 8)), path=dev(np.sort(np.argsort(rng.random((4, 8)), 1)[:, :5], 1)),
                          n_accept=dev(rng.integers(0, 6, 4)), gone=dev(rng.integers(0, 4, 2)),
                          q=torch.randn((4, T, 6, D), device="cuda", generator=g).to(DTYPES[dt]))
        self.buffers = {name: torch.empty_like(x) for name, x in self.first.items()}
        self.codes = torch.zeros((70, 2, 2, D), dtype=torch.int8, device="cuda")
        self.scales = torch.zeros((70, 2), device="cuda")

    def load(self, zero=False):
        for name, x in self.buffers.items():
            x.zero_() if zero else x.copy_(self.first[name])
        self.codes.zero_(), self.scales.zero_()

    def run(self, stream=None):
        b, page = self.buffers, self.page
        table, lens, refs, moves, count = kv.ibp_kv_fork(b["table"], b["lens"], b["refs"], b["parents"], page, stream=stream)
        kv.ibp_kv_copy(b["pool"], moves, count, stream=stream)
        kv.ibp_kv_summarize(b["pool"][0], table, lens, self.codes, self.scales, stream=stream)
        sparse = kv.ibp_sparse_attention(b["q"], b["pool"][0], b["pool"][1], table, lens, self.codes, self.scales, 4,
                                         stream=stream)
        state = kv.ibp_kv_accept(b["pool"], table, lens, refs, b["n_draft"], b["path"], b["n_accept"], stream=stream)
        state = kv.ibp_kv_free(*state, b["gone"], page, stream=stream)
        packed = kv.ibp_kv_compact(state[0], state[2], page, stream=stream)
        kv.ibp_kv_copy(b["pool"], packed[2], packed[3], stream=stream)
        return [table, lens, refs, moves, count, *sparse, *state, *packed, b["pool"], self.codes, self.scales]


NAMES = ["table", "lens", "refs", "moves", "count", "out", "lse", "pages", "accepted and freed table", "lens", "refs",
         "packed table", "refs", "moves", "count", "pool", "codes", "scales"]


def unlike(got, want):
    """What differs, by name."""
    return [f"{name} at {(a != b).nonzero()[0].tolist()}: {a[a != b][:4].tolist()} for {b[a != b][:4].tolist()}"
            for name, a, b in zip(NAMES, got, want) if not torch.equal(a, b)]


def test_every_call_goes_to_its_stream():
    """The stream holds the inputs back: a call that went elsewhere would read zeros."""
    step, side = Step(1), torch.cuda.Stream()
    step.load()
    want = [x.clone() for x in step.run()]
    step.load(zero=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        step.load()
    got = step.run(stream=side)
    side.synchronize()
    assert not unlike(got, want)
    step.load(zero=True)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        step.load()
        got = step.run()  # the current stream
    side.synchronize()
    assert not unlike(got, want)


def test_every_call_in_a_graph():
    steps = [Step(2), Step(3)]
    wants = []
    for s in steps:
        s.load()
        wants.append([x.clone() for x in s.run()])
    held, inputs, graph = steps[0], [s.first for s in steps], torch.cuda.CUDAGraph()
    held.load()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = held.run()
    for first, want in [*zip(inputs, wants)] * 2:  # other inputs on every replay
        held.first = first
        held.load()
        graph.replay()
        assert not unlike(got, want)


def test_calls_from_two_host_threads():
    """Each thread on its own stream, with forms of its own and a form they share."""
    forms = [dict(), dict(lens=(200, 90, 43), T=3, D=128, dt="f16")]
    wants = {}
    for i, f in enumerate(forms):
        step = Step(5, **f)
        step.load()
        wants[i] = [x.clone() for x in step.run()]
    c = Cache([700, 60, 1300], 4, 40, 4, 16, 128)
    tree = c.tree()
    torch.cuda.synchronize()
    wrong = []

    def work(mine):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                steps = {i: Step(5, **forms[i]) for i in (mine, 0)}
                for _ in range(60):
                    for i, step in steps.items():
                        step.load()
                        wrong.extend(unlike(step.run(), wants[i]))
                    if not all(torch.equal(a, b) for a, b in zip(c.tree(), tree)):
                        wrong.append("tree")
        except Exception as e:  # shown by the assertion below
            wrong.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not wrong


def test_a_first_call_inside_a_capture(monkeypatch):
    """The device's status word is made outside of captures: a first call inside one is
    refused and leaves the capture whole; ibp_kv_get_status makes the word."""
    c = Cache([300, 40], 2, 2, 2, 16, 64)
    want = c.tree()
    err(ibp.IBP_OK)
    monkeypatch.setattr(kv, "_status_words", {})
    a, more, graph = torch.ones(8, device="cuda"), dev(np.full(2, 7)), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = a + 1
        with pytest.raises(RuntimeError, match="ibp_kv_get_status"):
            c.tree()
    graph.replay()
    assert (b == 2).all()
    own, graph = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.tree(status=own)
    graph.replay()
    assert torch.equal(got[0], want[0]) and own.item() == 0 and not kv._status_words
    assert kv.ibp_kv_get_status() == ibp.IBP_OK and len(kv._status_words) == 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = c.tree(n_draft=more)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    err(ibp.IBP_ERANGE)


# ---------------------------------------------------------------------------
# Refusals


def test_misaligned_pointers_are_refused():
    """Every 32-bit array of the C entry points, two bytes off its alignment, is refused
    before a launch."""
    lib = kv._load()
    c = Cache([40, 20], 1, 2, 2, 16, 64)
    none = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    room = [torch.zeros(4096, dtype=torch.int32, device="cuda") for _ in range(13)]
    table, lens, refs, parents, t_out, l_out, r_out, moves, count, ws, word, path, lse = [r.data_ptr() for r in room]
    n = len(c.np_refs)
    kp, vp = kv._as_pages("k", c.k), kv._as_pages("v", c.v)
    kp.data, vp.data = c.k.data_ptr(), c.v.data_ptr()
    q, out = c.q.data_ptr(), torch.empty_like(c.q)
    codes, scales = c.codes, c.scales
    rows = (*c.q.stride()[:3], 1, 4)
    size = 4096 * 4

    def seqs(a):
        return kv._Seqs(a["table"], a["lens"], 2, c.table.shape[1])

    calls = {
        "fork": (lambda a: lib.ibp_kv_fork(seqs(a), 16, a["refs"], n, a["parents"], 2, a["t_out"], a["l_out"], a["r_out"],
                                           a["moves"], a["count"], a["ws"], size, a["word"], none),
                 dict(table=table, lens=lens, refs=refs, parents=parents, t_out=t_out, l_out=l_out, r_out=r_out, moves=moves,
                      count=count, ws=ws, word=word)),
        "free": (lambda a: lib.ibp_kv_free(seqs(a), 16, a["refs"], n, a["rows"], 1, a["t_out"], a["l_out"], a["r_out"],
                                           a["word"], none),
                 dict(table=table, lens=lens, refs=refs, rows=parents, t_out=t_out, l_out=l_out, r_out=r_out, word=word)),
        "compact": (lambda a: lib.ibp_kv_compact(seqs(a), 16, a["refs"], n, a["t_out"], a["r_out"], a["moves"], a["count"],
                                                 a["ws"], size, a["word"], none),
                    dict(table=table, lens=lens, refs=refs, t_out=t_out, r_out=r_out, moves=moves, count=count, ws=ws,
                         word=word)),
        "copy": (lambda a: lib.ibp_kv_copy(kp, a["moves"], a["count"], 1, a["word"], none),
                 dict(moves=moves, count=count, word=word)),
        "accept": (lambda a: lib.ibp_kv_accept(kp, seqs(a), a["refs"], a["n_draft"], a["path"], a["n_accept"], 1, a["t_out"],
                                               a["l_out"], a["r_out"], a["word"], none),
                   dict(table=table, lens=lens, refs=refs, n_draft=parents, path=path, n_accept=count, t_out=t_out,
                        l_out=l_out, r_out=r_out, word=word)),
        "tree": (lambda a: lib.ibp_tree_attention(kp, vp, 0, seqs(a), q, *rows, a["n_draft"], a["mask"], 1.0, out.data_ptr(),
                                                  a["lse"], None, 0, a["word"], none),
                 dict(table=table, lens=lens, n_draft=parents, mask=path, lse=lse, word=word)),
        "summarize": (lambda a: lib.ibp_kv_summarize(kp, 0, seqs(a), a["first"], a["codes"], a["scales"], a["word"], none),
                      dict(table=table, lens=lens, first=parents, codes=codes.data_ptr(), scales=scales.data_ptr(),
                           word=word)),
        "sparse": (lambda a: lib.ibp_sparse_attention(kp, vp, 0, seqs(a), a["codes"], a["scales"], q, *rows, a["n_query"], 2,
                                                      1, 1, 1.0, out.data_ptr(), a["lse"], a["pages"], ws, size, a["word"],
                                                      none),
                   dict(table=table, lens=lens, n_query=parents, codes=codes.data_ptr(), scales=scales.data_ptr(), lse=lse,
                        pages=moves, word=word)),
    }
    for name, (call, args) in calls.items():
        assert call(args) == ibp.IBP_OK, name  # lengths, counts and lists of zeros: little to do
        for which in args:
            assert call({**args, which: args[which] + 2}) == ibp.IBP_EINVAL, (name, which)
            assert lib.ibp_last_error_detail(), (name, which)
    torch.cuda.synchronize()


def test_tables_of_no_pages():
    """Sequences whose table rows have no entries yet: every call takes them."""
    none, lens = torch.empty((3, 0), dtype=torch.int32, device="cuda"), dev(np.zeros(3))
    refs = dev(np.array([0, 2, 0, 1]))
    table, new, moves, count = kv.ibp_kv_compact(none, refs, 16)
    assert table.shape == (3, 0) and host(new).tolist() == [1, 2, 0, 0] and count.item() == 1
    assert host(moves)[0].tolist() == [3, 0, 16]
    assert host(kv.ibp_kv_fork(none, lens, refs, dev(np.array([0, 2])), 16)[2]).tolist() == [0, 2, 0, 1]
    assert host(kv.ibp_kv_free(none, lens, refs, dev(np.array([1])), 16)[2]).tolist() == [0, 2, 0, 1]
    c = Cache([40], 2, 2, 2, 16, 64, spare=1)
    q = c.q.repeat(3, 1, 1, 1)
    out, lse = kv.ibp_tree_attention(q, c.k, c.v, none, lens, n_draft=lens)
    assert not out.any() and (lse == -float("inf")).all()
    out, lse, pages = kv.ibp_sparse_attention(q, c.k, c.v, none, lens, c.codes, c.scales, 2, n_query=lens)
    assert not out.any() and (lse == -float("inf")).all() and (pages == -1).all()
    assert torch.equal(kv.ibp_kv_summarize(c.k, none, lens, c.codes, c.scales)[0], c.codes)
    pool_ = torch.zeros((4, 1, 16, 8), dtype=torch.float16, device="cuda")
    path = torch.zeros((3, 1), dtype=torch.int32, device="cuda")
    got = kv.ibp_kv_accept(pool_, none, lens, refs, lens, path, lens)
    assert host(got[1]).tolist() == [0, 0, 0] and host(got[2]).tolist() == [0, 2, 0, 1]


def test_a_backward_through_attention_is_an_error():
    c = Cache([300, 40], 2, 2, 2, 16, 64)
    want, sparse = c.tree(), c.sparse(3)
    assert not want[0].requires_grad
    c.q.requires_grad_()
    got = c.tree()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(RuntimeError, match="ibp_tree_attention has no backward"):
        got[0].float().sum().backward()
    got = c.sparse(3)
    assert torch.equal(got[0], sparse[0]) and torch.equal(got[2], sparse[2])
    with pytest.raises(RuntimeError, match="ibp_sparse_attention has no backward"):
        got[1].sum().backward()
    with torch.no_grad():
        assert not c.tree()[0].requires_grad


# ---------------------------------------------------------------------------
# Waits that run out


@pytest.mark.parametrize("lens,T,hk,G,page,D", [
    ([700, 60, 1300], 4, 40, 4, 16, 128),   # one row tile
    ([700, 2000], 40, 12, 5, 64, 64),       # two
])
def test_waits_that_run_out_end_the_call(lens, T, hk, G, page, D):
    """Every wait of the kernel has a limit.  Met, the kernel reports IBP_ETIMEOUT and ends, and
    the calls behind it are right; the limits here are met in ordinary work."""
    c = Cache(lens, T, hk, G, page, D)
    want = c.tree()
    err(ibp.IBP_OK)
    try:
        for limit in (0, 1, 300, 1000, 3000, 10000):
            kv.ibp_kv_set_wait_limit(limit)
            got = c.tree()
            code = kv.ibp_kv_get_status(raise_on_error=False)
            assert code == ibp.IBP_ETIMEOUT if limit == 0 else code in (ibp.IBP_OK, ibp.IBP_ETIMEOUT)
            if code == ibp.IBP_OK:
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert kv.ibp_kv_set_wait_limit() == limit
            got = c.tree()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            err(ibp.IBP_OK)
    finally:
        assert kv.ibp_kv_set_wait_limit() == kv.IBP_KV_WAIT_CYCLES
    assert kv.ibp_kv_set_wait_limit(1 << 40) == kv.IBP_KV_WAIT_CYCLES  # no more than the default
    assert kv.ibp_kv_set_wait_limit() == kv.IBP_KV_WAIT_CYCLES
