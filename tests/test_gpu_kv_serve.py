"""GPU tests of the caches in 4 bits, the verification of drafted tokens and the eviction
of cached ones, against the CPU oracle."""

import ctypes
import threading

import numpy as np
import pytest
import torch

from host_transfer_gb300 import ibp, kv
from oracle import kv_ref, kv_serve_ref as ref
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


def pages_of(n, h, t, w, dtype, layout):
    """Pages in one of three memory orders; the third has room between tokens, heads and pages."""
    if layout == "hnd":
        return torch.empty((n, h, t, w), dtype=dtype, device="cuda")
    if layout == "nhd":
        return torch.empty((n, t, h, w), dtype=dtype, device="cuda").transpose(1, 2)
    more = 16 if dtype == torch.uint8 else 3
    return torch.empty((n, h + 1, t + 1, w + more), dtype=dtype, device="cuda")[:, :h, :t, :w]


def cache4(n, h, t, dim, dt, layout, g, spread=1.0):
    """Random codes and scales of 5 significant bits."""
    codes = pages_of(n, h, t, dim // 2, torch.uint8, layout)
    codes.copy_(torch.randint(0, 256, codes.shape, generator=g, device="cuda", dtype=torch.uint8))
    scales = pages_of(n, h, t, dim // 32, DTYPES[dt], layout)
    five = torch.randint(16, 32, scales.shape, generator=g, device="cuda").float()
    scales.copy_(five * spread * 2.0 ** torch.randint(-10, -7, scales.shape, generator=g, device="cuda").float())
    return codes, scales


def decoded(pair):
    return ref.values(host(pair[0]), host(pair[1]))


def unheld(table, lens, n_pages, page):
    """True where no sequence holds the token of a page."""
    free = np.ones((n_pages, page), bool)
    for b, n in enumerate(lens):
        for p in range(int(n)):
            if 0 <= table[b, p // page] < n_pages:
                free[table[b, p // page], p % page] = False
    return torch.from_numpy(free).cuda()[:, None, :, None]


# ---------------------------------------------------------------------------
# Storing and loading


@pytest.mark.parametrize("layout", ["hnd", "nhd", "padded"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("B,T,heads,dim,page", [(1, 1, 1, 32, 1), (3, 1, 8, 128, 16), (4, 37, 3, 96, 7), (2, 130, 2, 256, 64),
                                                (5, 3, 2, 160, 24), (2, 20, 1, 64, 16)])
def test_store_and_load(B, T, heads, dim, page, dt, layout):
    rng = np.random.default_rng(B * 100 + T)
    lens = rng.integers(T, T + 50, B).astype(np.int32)
    n_pages = int((-(-lens // page)).sum()) + 2
    table, _ = tables(lens, page, n_pages, int(-(-lens.max() // page)) + 1, rng)
    n_new = rng.integers(0, T + 1, B).astype(np.int32) if T > 1 else None
    g = gen(T)
    k4, v4 = (cache4(n_pages, heads, page, dim, dt, layout, g) for _ in range(2))
    # rows of a fused projection, and rows that are not 16-byte aligned
    both = torch.randn((B, T, 2 * heads, dim), generator=g, device="cuda").to(DTYPES[dt])
    k, v = both[:, :, :heads], both[:, :, heads:]
    if layout == "padded":
        v = torch.randn((B, heads, T, dim + 1), generator=g, device="cuda").to(DTYPES[dt])[..., 1:].transpose(1, 2)
    want = [ref.store(host(x), host(c[0]), host(c[1]), table, lens, n_new, dt == "f16") for x, c in ((k, k4), (v, v4))]
    n_dev = None if n_new is None else dev(n_new)
    kv.ibp_kv4_store(k, v, k4, v4, dev(table), dev(lens), n_new=n_dev)
    for got, w in zip((k4, v4), want):
        assert np.array_equal(host(got[0]), w[0]) and np.array_equal(host(got[1]), w[1].astype(np.float32))
    got = kv.ibp_kv4_load(k4, v4, dev(table), dev(lens), T, n_load=n_dev)
    for x, w in zip(got, want):
        assert np.array_equal(host(x), ref.load(*w, table, lens, T, n_new))
    # everything that the sequences hold
    longest = int(lens.max())
    got = kv.ibp_kv4_load(k4, v4, dev(table), dev(lens), longest, n_load=dev(lens))
    for x, w in zip(got, want):
        assert np.array_equal(host(x), ref.load(*w, table, lens, longest, lens))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_store_special_values(dt):
    """Ties of scale and code, the type's smallest and largest values, infinities and NaN."""
    t = DTYPES[dt]
    tiny, huge = (2.0**-24, 65504.0) if dt == "f16" else (2.0**-133, float(torch.finfo(t).max))
    groups = [[7 * (1 + i / 32)] + [(j + 0.5) * (1 + i / 32) for j in range(-7, 7)] + [0] * 17 for i in range(32)]
    groups += [[0.0] * 32, [-0.0] * 32, [tiny] * 32, [tiny * i for i in range(32)], [huge, -huge] * 16,
               [2.0**-99 * i for i in range(32)], [7 * 2.0**-100] * 32, [6.5 * 2.0**-100] * 32, [7 * 2.0**-25] * 32,
               [float("inf")] + [1.0] * 31, [1.0] * 31 + [float("nan")], [-float("inf")] * 32, [1e-3, 1.0] * 16]
    x = torch.tensor(groups, dtype=torch.float32, device="cuda").to(t).reshape(1, 1, -1, 32)
    n = x.shape[2]
    k4, v4 = (cache4(1, n, 1, 32, dt, "hnd", gen(1)) for _ in range(2))
    table, lens = np.zeros((1, 1), np.int32), np.ones(1, np.int32)
    want = ref.store(host(x), host(k4[0]), host(k4[1]), table, lens, None, dt == "f16")
    kv.ibp_kv4_store(x, -x, k4, v4, dev(table), dev(lens))
    assert np.array_equal(host(k4[0]), want[0]) and np.array_equal(host(k4[1]), want[1].astype(np.float32), equal_nan=True)
    got, neg = kv.ibp_kv4_load(k4, v4, dev(table), dev(lens), 1)
    assert np.array_equal(host(got), ref.load(*want, table, lens, 1, None), equal_nan=True)
    fine = torch.isfinite(got)
    assert torch.equal(got[fine], -neg[fine])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_values_of_any_scale(dt):
    """All codes times all scales: the loaded values are the exact products where the type holds them."""
    t = DTYPES[dt]
    bits = torch.arange(65536, dtype=torch.int32, device="cuda").to(torch.int16)
    scales = bits.view(t).reshape(1, 1, 65536, 1)
    codes = torch.tensor([2 * i | (2 * i + 1) << 4 for i in range(8)] * 2, dtype=torch.uint8, device="cuda")
    codes = codes.expand(1, 1, 65536, 16).contiguous()
    got, _ = kv.ibp_kv4_load((codes, scales), (codes, scales), dev(np.zeros((1, 1))), dev(np.array([65536])), 65536)
    with np.errstate(invalid="ignore"):
        s = host(scales)[0, 0, :, 0].astype(np.float64)
    if dt == "bf16":  # the 3 lowest bits are not read; from 2^122 on: NaN
        with np.errstate(invalid="ignore"):
            s = host((bits & -8).view(t)).astype(np.float64)
        s[~(np.abs(s) < 2.0**122)] = np.nan
    with np.errstate(invalid="ignore", over="ignore"):
        want = np.arange(-8, 8)[None] * s[:, None]
        want = want.astype(np.float16).astype(np.float64) if dt == "f16" else want
    assert np.array_equal(host(got)[0, :, 0, :16].astype(np.float64), want, equal_nan=True)


def test_store_and_load_report_what_is_out_of_range():
    g = gen(5)
    k4, v4 = (cache4(4, 1, 16, 64, "bf16", "hnd", g) for _ in range(2))
    x = torch.randn((2, 3, 1, 64), generator=g, device="cuda").bfloat16()
    for table, lens, n_new in (([[0, 9], [1, 2]], [18, 20], None),       # a page id
                               ([[0, 3], [1, 2]], [2, 20], None),        # a position below 0
                               ([[0, 3], [1, 2]], [20, 20], [3, 7]),     # more rows than there are
                               ([[0, 3], [1, 2]], [20, 20], [-1, 3]),
                               ([[0, 3], [1, 2]], [20, 40], None)):      # a length beyond the table
        table, lens = np.array(table, np.int32), np.array(lens, np.int32)
        cut = np.minimum(lens, 32)
        want = ref.store(host(x), host(k4[0]), host(k4[1]), table, cut, n_new, False)
        n_dev = None if n_new is None else dev(np.array(n_new))
        kv.ibp_kv4_store(x, x, k4, v4, dev(table), dev(lens), n_new=n_dev)
        err(ibp.IBP_ERANGE)
        assert np.array_equal(host(k4[0]), want[0]) and np.array_equal(host(k4[1]), want[1].astype(np.float32))
        got, _ = kv.ibp_kv4_load(k4, v4, dev(table), dev(lens), 3, n_load=n_dev)
        err(ibp.IBP_ERANGE)
        assert np.array_equal(host(got), ref.load(*want, table, cut, 3, n_new))


def test_store_past_32_bits():
    """A pool whose last page lies more than 2^32 bytes in."""
    page, n = 64, 9
    codes = torch.empty((n, 1, page, 64), dtype=torch.uint8, device="cuda")
    room = torch.empty((1 << 32) + (1 << 29), dtype=torch.uint8, device="cuda")
    codes = room.as_strided((n, 1, page, 64), (1 << 29, 64 * page, 64, 1))
    scales = torch.zeros((n, 1, page, 4), dtype=torch.bfloat16, device="cuda")
    x = torch.randn((1, 3, 1, 128), device="cuda", generator=gen(2)).bfloat16()
    table, lens = dev(np.array([[8, 0]])), dev(np.array([3]))
    kv.ibp_kv4_store(x, x, (codes, scales), (codes, scales), table, lens)
    got, _ = kv.ibp_kv4_load((codes, scales), (codes, scales), table, lens, 3)
    want = ref.values(*[y.astype(z) for y, z in zip((ref.pack(ref.quantise(host(x), False)[0]), ref.quantise(host(x), False)[1]),
                                                  (np.uint8, np.float64))])
    assert np.array_equal(host(got), want)
    q = torch.randn((1, 1, 1, 128), device="cuda", generator=gen(3)).bfloat16()
    out, lse = kv.ibp_kv4_attention(q, (codes, scales), (codes, scales), table, lens)
    pages = np.zeros((n, 1, page, 128))
    pages[8, 0, :3] = want[0, :, 0]
    check_attention(out, lse, *kv_ref.tree_attention(host(q), pages, pages, np.array([[8, 0]]), [3]), "bf16")


# ---------------------------------------------------------------------------
# Attention


class Cache:
    def __init__(self, lens, T, hk, G, page, D, dt="bf16", layout="hnd", seed=0, spare=3, mask=False, spread=1.0):
        rng = np.random.default_rng(seed)
        self.np_lens = np.array(lens, np.int32)
        n_pages = int((-(-self.np_lens // page)).sum()) + spare
        width = max(1, -(-int(max(lens)) // page)) + 1
        self.np_table, self.np_refs = tables(lens, page, n_pages, width, rng)
        g = gen(seed)
        self.k, self.v = (cache4(n_pages, hk, page, D, dt, layout, g, spread) for _ in range(2))
        self.np_k, self.np_v = decoded(self.k), decoded(self.v)
        # what no sequence holds must not matter
        free = unheld(self.np_table, self.np_lens, n_pages, page)
        for x in (self.k, self.v):
            x[1].masked_fill_(free, float("nan"))
            x[0].masked_fill_(free, 0xF3)
        self.q = torch.randn((len(lens), T, hk * G, D), device="cuda", generator=g).to(DTYPES[dt])
        self.table, self.lens, self.refs = dev(self.np_table), dev(self.np_lens), dev(self.np_refs)
        self.dt, self.page, self.np_mask, self.mask = dt, page, None, None
        if mask:
            bits = rng.integers(0, 2**32, (len(lens), T, -(-T // 32)), dtype=np.uint32)
            bits[:, 0] = 0  # a row that sees no drafted token
            self.np_mask, self.mask = bits, dev(bits.view(np.int32))

    def attend(self, **kw):
        return kv.ibp_kv4_attention(self.q, self.k, self.v, self.table, self.lens, mask=self.mask, **kw)

    def want(self, n_draft=None, scale=None):
        return kv_ref.tree_attention(host(self.q), self.np_k, self.np_v, self.np_table, self.np_lens, self.np_mask, n_draft, scale)

    def check(self, **kw):
        n_draft = kw.get("n_draft")
        got = self.attend(**{**kw, **({} if n_draft is None else {"n_draft": dev(n_draft)})})
        check_attention(*got, *self.want(n_draft, kw.get("scale")), self.dt)


@pytest.mark.parametrize("layout", ["hnd", "nhd", "padded"])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D,mask", [
    ([1], 1, 1, 1, 16, 32, False), ([17, 5, 300], 1, 2, 4, 16, 64, False), ([40, 33], 1, 1, 9, 48, 96, False),
    ([700, 1, 95], 1, 2, 3, 7, 128, False), ([200, 64], 5, 2, 2, 64, 128, True), ([90, 41, 41], 41, 1, 1, 24, 160, True),
    ([130], 33, 1, 2, 16, 256, True), ([33, 70], 3, 3, 1, 1, 224, False), ([260, 3], 3, 1, 16, 32, 128, True),
])
def test_attention(lens, T, hk, G, page, D, mask, dt, layout):
    Cache(lens, T, hk, G, page, D, dt, layout, seed=T, mask=mask).check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D", [
    ([3000], 1, 1, 4, 16, 128), ([9000, 200, 4100], 1, 1, 2, 64, 64), ([5000] * 3, 2, 1, 3, 24, 256),
    ([20000, 7000], 1, 2, 1, 128, 128), ([2500, 1024, 1023, 0, 4096] * 40, 1, 2, 2, 64, 64),
])
def test_attention_over_long_caches(lens, T, hk, G, page, D, dt):
    """Shares of a cluster of CTAs, and chunks joined by a second kernel."""
    c = Cache(lens[:5], T, hk, G, page, D, dt, seed=len(lens))
    if len(lens) > 5:  # the same five sequences over and over
        n = len(lens) // 5
        c.np_lens, c.np_table = np.tile(c.np_lens, n), np.tile(c.np_table, (n, 1))
        c.lens, c.table, c.q = c.lens.repeat(n), c.table.repeat(n, 1), c.q.repeat(n, 1, 1, 1)
        one = kv_ref.tree_attention(host(c.q[:5]), c.np_k, c.np_v, c.np_table[:5], c.np_lens[:5], n_draft=[1, 1, 1, 0, 1])
        live = dev(np.array([1, 1, 1, 0, 1] * n))
        check_attention(*c.attend(n_draft=live), *(np.tile(x, (n,) + (1,) * (x.ndim - 1)) for x in one), dt)
    else:
        c.check()


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D,mask", [
    ([300, 290] * 3, 17, 2, 8, 64, 128, True), ([200, 141, 141, 150] * 2, 141, 3, 1, 7, 64, False),
    ([170] * 12, 130, 2, 1, 16, 96, True), ([90, 700, 41] * 4, 40, 4, 1, 24, 32, True),
    ([300, 290] * 2, 40, 2, 8, 64, 128, True), ([310, 305, 301], 300, 2, 1, 5, 64, True),
    ([150, 160, 100], 37, 3, 8, 16, 96, False), ([300, 290], 66, 2, 8, 64, 128, True),
    ([600, 641], 600, 1, 1, 7, 64, False), ([310, 305, 301], 130, 2, 4, 5, 96, True), ([170] * 40, 9, 2, 2, 16, 128, True),
])
def test_attention_of_many_rows(lens, T, hk, G, page, D, mask, dt):
    """Calls for the tensor cores: on codes, and (above 512 rows) decoded once."""
    c = Cache(lens, T, hk, G, page, D, dt, seed=T, mask=mask)
    B = len(lens)
    assert -(-max(lens) // 128) * B * hk * -(-T * G // 16) >= 304, "work enough for the tensor cores"
    live = np.array([T - (i % 3) for i in range(B)], np.int32)
    c.check(n_draft=live)


@pytest.mark.parametrize("lens,T,n_draft", [([0, 5, 2], 3, None), ([0, 0, 0], 1, None), ([9, 9, 9], 4, [0, 5, -1]),
                                            ([40, 3, 17], 20, [20, 20, 0])])
@pytest.mark.parametrize("G,D", [(2, 64), (9, 128)])
def test_rows_that_see_nothing(lens, T, n_draft, G, D):
    c = Cache(lens, T, 2, G, 16, D, seed=3)
    got = c.attend(n_draft=None if n_draft is None else dev(np.array(n_draft)))
    cut = None if n_draft is None else np.clip(n_draft, 0, T)
    check_attention(*got, *c.want(cut), "bf16")
    live = [T] * 3 if n_draft is None else n_draft
    err(ibp.IBP_ERANGE if any(not 0 <= n <= min(T, m) for n, m in zip(live, lens)) else ibp.IBP_OK)


def test_attention_sees_bad_pages_as_zeros():
    for T, G in ((2, 3), (60, 8)):
        c = Cache([3000, 2000, 900], T, 2, G, 16, 64, seed=4)
        c.np_table[0, 3], c.np_table[1, 60], c.np_table[2, 0] = -1, 10**6, c.np_k.shape[0]
        c.table = dev(c.np_table)
        c.check()
        err(ibp.IBP_ERANGE)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,hk,G,page", [(3, 1, 2, 16), (7, 2, 1, 24), (13, 1, 4, 16), (70, 8, 4, 16)])
def test_values_that_are_not_finite_reach_only_the_rows_that_see_them(T, hk, G, page, dt):
    lens = [T + 30, T + 900, T]
    c = Cache(lens, T, hk, G, page, 64, dt, seed=T)
    rng = np.random.default_rng(7)
    bits = np.zeros((3, T, -(-T // 32)), np.uint32)
    sees = rng.random((3, T, T)) < 0.5
    odd = T - 2
    sees[:, :, odd] = np.arange(T) % 2 == 1
    for t in range(T):
        for i in range(T):
            bits[:, t, i // 32] |= (sees[:, t, i].astype(np.uint32) << np.uint32(i % 32)).astype(np.uint32)
    c.np_mask, c.mask = bits, dev(bits.view(np.int32))
    clean = c.attend()
    check_attention(*clean, *c.want(), dt)
    for bad in (float("nan"), float("inf"), 9000.0 if dt == "f16" else 2.0**125):
        k, v = (c.k[0].clone(), c.k[1].clone()), (c.v[0].clone(), c.v[1].clone())
        for b in range(3):
            pos = lens[b] - T + odd
            at = int(c.np_table[b, pos // page]), hk - 1, pos % page
            v[1][at] = bad
            v[0][at] = 0x08  # -8 and 0
        out, lse = kv.ibp_kv4_attention(c.q, k, v, c.table, c.lens, mask=c.mask)
        hidden = torch.from_numpy(~sees[:, :, odd]).cuda()
        first = hk * G - G
        assert torch.equal(out[:, :, :first], clean[0][:, :, :first]) and torch.equal(lse, clean[1])
        assert torch.equal(out[:, :, first:][hidden], clean[0][:, :, first:][hidden])
        seen = out[:, :, first:][~hidden]
        assert not torch.isfinite(seen[..., 1::2]).all() or bad == 9000.0  # code 0: -8 times the scale
        # keys: only the rows that see them
        for b in range(3):
            pos = lens[b] - T + odd
            k[1][int(c.np_table[b, pos // page]), hk - 1, pos % page] = bad
        if bad != bad:
            out, lse = kv.ibp_kv4_attention(c.q, k, c.v, c.table, c.lens, mask=c.mask)
            assert torch.equal(out[:, :, first:][hidden], clean[0][:, :, first:][hidden])
            assert torch.isnan(out[:, :, first:][~hidden]).all()


@pytest.mark.parametrize("scale", [-0.5, 0.0, 3.0])
@pytest.mark.parametrize("T,hk,G", [(2, 2, 2), (33, 8, 8)])
def test_scales_of_any_sign(scale, T, hk, G):
    Cache([90, 64, 200], T, hk, G, 16, 64, seed=8).check(scale=scale)


def test_large_scores():
    """Single precision ends at 2^-126 (its exponential gives 0 below): a probability that
    is smaller is lost whole, so an output whose large probabilities meet zeros is off by up
    to that for each of the 200 tokens, times the largest value.  The checker's
    bound has u times the mean, which is raised by as much over u."""
    for dt, u in (("bf16", 2.0**-8), ("f16", 2.0**-11)):
        c = Cache([90, 64, 200], 3, 2, 2, 16, 64, dt, seed=8, spread=64.0)
        out, lse, mean, top = c.want(scale=8.0)
        floor = 200 * 2.0**-126 * np.nanmax(np.abs(c.np_v)) / u
        check_attention(*c.attend(scale=8.0), out, lse, mean + floor, top, dt)


def test_queries_by_strides_and_given_results():
    c = Cache([200, 77], 4, 2, 3, 16, 96, seed=11)
    wide = torch.randn((2, 6, 5, 100), device="cuda", generator=gen(1)).bfloat16()
    c.q = wide.transpose(1, 2)[:, :4, :, 2:98]
    c.check()
    out = torch.empty((2, 4, 6, 96), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((2, 4, 6), device="cuda")
    got = c.attend(out=out, lse=lse)
    assert got[0] is out and got[1] is lse


def test_many_rows_equal_the_16_bit_call():
    """What the codes stand for, loaded into pages of 16 bits, gives the same attention."""
    c = Cache([1500, 1700, 800, 90], 64, 8, 4, 64, 128, "bf16", seed=12)
    n = 1700
    k, v = kv.ibp_kv4_load(c.k, c.v, c.table, c.lens, n, n_load=c.lens)
    pages = [torch.zeros((4 * 14, 8, 128, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.arange(56, dtype=torch.int32, device="cuda").reshape(4, 14)
    for x, p in zip((k, v), pages):
        x = torch.nn.functional.pad(x, (0, 0, 0, 0, 0, 14 * 128 - n))
        p.copy_(x.reshape(56, 128, 8, 128).transpose(1, 2))
    want = kv.ibp_tree_attention(c.q, *pages, table, c.lens)
    got = c.attend()
    # the same products; the number of CTAs, and so the order of the sums, may differ
    assert (got[0].float() - want[0].float()).abs().max() <= 2.0**-7 * want[0].float().abs().max()
    assert (got[1] - want[1]).abs().max() < 1e-4


# ---------------------------------------------------------------------------
# Verification


def draft(B, T, V, tree, seed, sharp=2.0, off=0.7, certain=False):
    rng = np.random.default_rng(seed)

    def softmax(x):
        e = np.exp(x - x.max(-1, keepdims=True))
        return (e / e.sum(-1, keepdims=True)).astype(np.float32)

    logits = rng.normal(size=(B, T + 1, V)) * sharp
    q, p = softmax(logits[:, :T]), softmax(logits + rng.normal(size=logits.shape) * off)
    parents = None
    if tree:
        parents = np.maximum(np.arange(T) - rng.integers(1, 5, (B, T)), -1).astype(np.int32)
    tokens = np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(T):
            row = q[b, t if parents is None else parents[b, t] + 1].astype(np.float64)
            tokens[b, t] = row.argmax() if certain and rng.random() < 0.5 else rng.choice(V, p=row / row.sum())
    u = rng.random((B, T + 1)).astype(np.float32)
    u = np.minimum(u, np.float32(1 - 2.0**-24))
    return p, tokens, u, None if certain else q, parents


def run_verify(p, tokens, u, q=None, parents=None, n_draft=None):
    got = kv.ibp_kv_verify(dev(p, torch.float32), dev(tokens), dev(u, torch.float32),
                           None if q is None else dev(q, torch.float32), None if parents is None else dev(parents),
                           None if n_draft is None else dev(n_draft))
    want = ref.verify(p, tokens, u, q, parents, n_draft)
    for x, y, name in zip(got, want, ("path", "n_accept", "token")):
        assert np.array_equal(host(x), y), name
    err(ibp.IBP_ERANGE if want[3] else ibp.IBP_OK)
    return want


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("B,T,V", [(1, 1, 1), (2, 1, 2), (5, 4, 33), (17, 9, 1000), (3, 24, 4097), (4, 6, 16384), (2, 5, 40001),
                                   (9, 15, 513), (2, 3, 262144)])
def test_verify(B, T, V, tree, certain):
    p, tokens, u, q, parents = draft(B, T, V, tree, B + T + V, certain=certain)
    run_verify(p, tokens, u, q, parents)


@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("V", [5, 300, 20000])
def test_verify_many_siblings(V, certain):
    """All tokens tried behind the context, most of them rejected, some of them alike."""
    rng = np.random.default_rng(V)
    p, _, u, q, _ = draft(6, 12, V, False, V + 1, certain=False, off=3.0)
    tokens = rng.integers(0, min(V, 8), (6, 12)).astype(np.int32)
    parents = np.full((6, 12), -1, np.int32)
    parents[3:, 6:] = 2
    u[:, :12] = 1 - u[:, :12] * 1e-3
    run_verify(p, tokens, u, None if certain else q, parents)


@pytest.mark.parametrize("V", [8, 5000, 20000])
def test_verify_rejections_on_both_sides_of_an_acceptance(V):
    """A token is accepted behind a rejected one, and then its child with the same token is
    rejected: the rejected tokens are listed anew while the first list may still be read."""
    B, T = 40, 12
    rng = np.random.default_rng(V)
    p = rng.random((B, T + 1, V)).astype(np.float32) ** 4
    p /= p.sum(-1, keepdims=True)
    # four times: a token rejected, one accepted, and that one again behind itself rejected
    tokens = np.tile(np.array([1, 2, 2, 1, 3, 3], np.int32), (B, T // 6))
    parents = np.tile(np.array([[-1, -1, 1, 1, 1, 4, 4, 4, 7, 7, 7, 10]], np.int32), (B, 1))
    u = np.tile(np.array([1, 0, 1], np.float32), (B, T // 3))
    u = np.concatenate([u, rng.random((B, 1), np.float32)], 1)
    assert (run_verify(p, tokens, u, None, parents)[1] == 4).all()


def test_verify_no_drafts_and_many():
    p, tokens, u, q, _ = draft(3, 5, 100, False, 1)
    for n in ([0, 0, 0], [5, 2, 0], [7, -1, 3]):
        run_verify(p, tokens, u, q, None, np.array(n, np.int32))
    run_verify(p[:, :1], tokens[:, :0], u[:, :1])
    p, tokens, u, q, parents = draft(2, 1024, 16, True, 2)
    run_verify(p, tokens, u, q, parents)
    run_verify(p, tokens, u, q)


def test_verify_equal_distributions_and_empty_rows():
    """Where nothing is left of the target's probabilities the rest stays; rows of zeros draw nothing."""
    p, tokens, u, q, _ = draft(4, 3, 600, False, 3)
    q = p[:, :3].copy()
    u[:] = [[0.5, 1.0, 1.5, 0.25], [1.0, 0, 0, 0.999], [2.0, 0, 0, 0], [0, 0, 0, 1.0]]
    run_verify(p, tokens, u, q)
    run_verify(np.zeros_like(p), tokens, u, q)
    run_verify(p, tokens, u, np.zeros_like(q))
    run_verify(p, tokens, np.zeros_like(u), q)


def test_verify_values_out_of_the_ordinary():
    p, tokens, u, q, parents = draft(6, 6, 700, True, 4)
    p[0, :, ::7] = np.nan
    p[1] *= 1000
    p[2] = -p[2]
    p[3, :, 5] = np.inf
    p[4] *= 1e-12
    q[5, :, ::3] = np.nan
    q[0] *= -1
    u[1, 2], u[2, 6], u[3, 6], u[4, 6] = np.nan, np.nan, np.inf, -1.0
    run_verify(p, tokens, u, q, parents)


def test_verify_reports_what_is_out_of_range():
    p, tokens, u, q, parents = draft(4, 6, 50, True, 5)
    for b, (t, x, r) in enumerate([(0, 50, -1), (2, -1, 1), (3, 4, 3), (5, 7, -2)]):
        tokens[b, t], parents[b, t] = x, r
    run_verify(p, tokens, u, q, parents)


def test_verify_rows_by_strides():
    p, tokens, u, q, _ = draft(3, 4, 501, False, 6)
    wide_p = torch.full((3, 5, 510), float("nan"), device="cuda")
    wide_p[..., 3:504] = dev(p, torch.float32)
    wide_q = dev(q, torch.float32).transpose(0, 1).contiguous().transpose(0, 1)
    got = kv.ibp_kv_verify(wide_p[..., 3:504], dev(tokens), dev(u, torch.float32), wide_q)
    assert all(np.array_equal(host(x), y) for x, y in zip(got, ref.verify(p, tokens, u, q)))


# ---------------------------------------------------------------------------
# Accumulated weight and eviction


def check_weigh(got, want, top, lse, rows, was, decay):
    """Each term's exponent is off by the score's error, (dim + 8) 2^-23 of the largest sum of
    |q k| (dim <= 256), and by 2^-22 of |s| + |lse|, itself at most the same sum and
    the largest lse; the exponential by 2^-21, the sums by 2^-24 a row and step."""
    fine = np.abs(lse[np.isfinite(lse)]).max() if np.isfinite(lse).any() else 0.0
    rel = 264 * 2.0**-23 * top + 2.0**-22 * (top + fine) * 1.5 + 2.0**-21 + rows * 2.0**-24
    tol = rel * np.abs(want) + 2.0**-22 * np.abs(decay * was) + 1e-30
    off = np.abs(host(got).astype(np.float64) - want) - tol
    assert (off <= 0).all(), f"off by {off.max():.3g} beyond the bound"


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("four", [True, False])
@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("lens,T,hk,G,page,D,mask", [
    ([1], 1, 1, 1, 16, 32, False), ([70, 0, 33], 1, 2, 4, 16, 64, False), ([300, 17], 1, 8, 1, 7, 128, False),
    ([100, 64, 80], 5, 3, 2, 24, 96, True), ([90, 41], 41, 1, 3, 64, 160, True), ([60], 7, 12, 2, 16, 256, False),
    ([130, 200], 33, 9, 1, 1, 128, True), ([500], 2, 1, 9, 16, 192, False),
    # the tensor cores: fewer heads than CTAs, more, a head's blocks shared out
    ([300, 90], 70, 3, 1, 16, 64, False), ([700], 40, 1, 8, 24, 128, True), ([120, 300], 17, 10, 4, 7, 96, True),
    ([0, 600], 64, 8, 1, 64, 128, False), ([260], 130, 2, 2, 16, 32, True),
    # work for clusters of two and of four
    ([250, 0, 190, 97] * 5, 21, 1, 4, 16, 64, True), ([120, 260] * 5, 90, 3, 1, 16, 128, False),
    ([180, 256, 33] * 6, 35, 1, 4, 16, 64, False), ([270, 140] * 5, 70, 5, 2, 24, 128, True),
])
def test_weigh(lens, T, hk, G, page, D, mask, dt, four, inplace):
    c = Cache(lens, T, hk, G, page, D, dt, seed=D + T, mask=mask)
    n_draft = np.array([max(0, min(T - i, n)) for i, n in enumerate(lens)], np.int32)
    if four:
        keys, np_keys = c.k, c.np_k
    else:
        np_keys = c.np_k
        keys = torch.from_numpy(np_keys).to("cuda", DTYPES[dt])
        keys.masked_fill_(unheld(c.np_table, c.np_lens, keys.shape[0], page), float("nan"))
    _, lse, _, _ = c.want(n_draft)
    lse = lse.astype(np.float32)
    rng = np.random.default_rng(1)
    width = c.np_table.shape[1] * page + 5
    was = rng.random((len(lens), width)).astype(np.float32)
    w = dev(was, torch.float32)
    want, top = ref.weigh(host(c.q), np_keys, c.np_table, c.np_lens, lse, was, c.np_mask, n_draft, decay=0.75)
    got = kv.ibp_kv_weigh(c.q, keys, c.table, c.lens, dev(lse, torch.float32), w, mask=c.mask, n_draft=dev(n_draft),
                          decay=0.75, inplace=inplace)
    assert (got.data_ptr() == w.data_ptr()) == inplace
    check_weigh(got, want, top, lse, T * hk * G, was, 0.75)
    for b, n in enumerate(lens):
        assert np.array_equal(host(got)[b, n:], was[b, n:])


def test_weights_sum_to_the_rows():
    """The weights that a step gives add up to one for each query and head."""
    c = Cache([5000, 4000], 3, 4, 8, 64, 128, seed=2)
    _, lse = c.attend()
    for decay in (0.0, 1.0):
        w = kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, torch.zeros((2, 5056), device="cuda"), decay=decay)
        assert torch.allclose(w.double().sum(1), torch.full((2,), 96.0, dtype=torch.float64, device="cuda"), rtol=1e-4)


def test_weigh_reports_what_is_out_of_range():
    c = Cache([100, 64], 2, 2, 2, 16, 64, seed=6)
    _, lse = c.attend()
    was = np.ones((2, 80), np.float32)
    got = kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, dev(was, torch.float32))  # the first is longer than the width
    want, top = ref.weigh(host(c.q), c.np_k, c.np_table, c.np_lens, host(lse), was)
    check_weigh(got, want, top, host(lse), 8, was, 1.0)
    err(ibp.IBP_ERANGE)
    c.np_table[0, 2] = -5
    was = np.ones((2, 112), np.float32)
    got = kv.ibp_kv_weigh(c.q, c.k, dev(c.np_table), c.lens, lse, dev(was, torch.float32))
    want, top = ref.weigh(host(c.q), c.np_k, c.np_table, c.np_lens, host(lse), was)
    check_weigh(got, want, top, host(lse), 8, was, 1.0)
    err(ibp.IBP_ERANGE)


def run_evict(w, lens, budget, first, last):
    want = ref.evict(w, lens, budget, first, last)
    got = kv.ibp_kv_evict(dev(w, torch.float32), dev(np.array(lens)), budget, keep_first=first, keep_last=last)
    for x, y, name in zip(got, want, ("path", "n_draft", "n_keep", "weights")):
        assert np.array_equal(host(x), y, equal_nan=x.is_floating_point()), name


@pytest.mark.parametrize("B,width,budget,first,last", [
    (1, 1, 1, 0, 0), (3, 40, 10, 2, 3), (4, 33, 32, 16, 16), (5, 700, 699, 0, 1), (2, 2048, 100, 4, 50), (3, 2049, 1024, 0, 0),
    (2, 9001, 1, 0, 0), (2, 9001, 9000, 4000, 5000), (3, 70000, 8192, 4, 1024), (2, 5000, 6000, 1, 1), (40, 300, 64, 0, 64),
])
@pytest.mark.parametrize("values", ["spread", "few", "equal", "odd"])
def test_evict(B, width, budget, first, last, values):
    rng = np.random.default_rng(width + budget)
    w = np.exp(rng.normal(size=(B, width)) * 3).astype(np.float32)
    if values == "few":
        w = rng.integers(0, 3, w.shape).astype(np.float32)
    elif values == "equal":
        w[:] = 0.25
    elif values == "odd":
        w[rng.random(w.shape) < 0.2] = np.nan
        w[rng.random(w.shape) < 0.1] = np.inf
        w[rng.random(w.shape) < 0.1] = -np.inf
        w[rng.random(w.shape) < 0.2] = -0.0
        w[rng.random(w.shape) < 0.2] = 0.0
        w[rng.random(w.shape) < 0.1] = np.float32(1e-42)
    lens = [width, *rng.integers(0, width + 1, B - 1).tolist()]
    run_evict(w, lens, budget, first, last)


def test_evict_lengths_beyond_the_weights():
    w = np.arange(60, dtype=np.float32).reshape(2, 30)
    want = ref.evict(w, [30, 0], 10, 1, 1)
    got = kv.ibp_kv_evict(dev(w, torch.float32), dev(np.array([31, -4])), 10, keep_first=1, keep_last=1)
    assert all(np.array_equal(host(x), y) for x, y in zip(got, want))
    err(ibp.IBP_ERANGE)


# ---------------------------------------------------------------------------
# Together


def pools_of(pair):
    return pair[0][None], pair[1][None]


def test_a_step_of_all_of_them():
    """Store drafted tokens, attend to the tree, verify, keep what is accepted, weigh, evict
    and attend again: the same cache as the oracle's after every step."""
    B, T, hk, G, page, D, budget = 4, 6, 2, 2, 16, 64, 80
    c = Cache([100, 60, 130, 90], 1, hk, G, page, D, seed=20, spare=9)
    rng = np.random.default_rng(21)
    # every sequence gets room for its draft
    lens = c.np_lens + T
    table, refs = c.np_table.copy(), c.np_refs.copy()
    table = np.concatenate([table, np.full((B, 2), -1, np.int32)], 1)
    for b in range(B):
        for p in range(-(-int(c.np_lens[b]) // page), -(-int(lens[b]) // page)):
            table[b, p] = int(np.flatnonzero(refs == 0)[0])
            refs[table[b, p]] = 1
    t_table, t_lens, t_refs = dev(table), dev(lens), dev(refs)
    g = gen(22)
    k, v, q = (torch.randn((B, T, h, D), generator=g, device="cuda").bfloat16() for h in (hk, hk, hk * G))
    caches = [[host(x) for x in c.k], [host(x) for x in c.v]]
    caches = [list(ref.store(host(x), *y, table, lens, None, False)) for x, y in zip((k, v), caches)]
    kv.ibp_kv4_store(k, v, c.k, c.v, t_table, t_lens)
    p, tokens, u, dist, parents = draft(B, T, 300, True, 23)
    bits = np.zeros((B, T, 1), np.uint32)
    for b in range(B):
        for t in range(T):
            bits[b, t, 0] = (1 << t) | (bits[b, parents[b, t], 0] if parents[b, t] >= 0 else 0)
    out, lse = kv.ibp_kv4_attention(q, c.k, c.v, t_table, t_lens, mask=dev(bits.view(np.int32)))
    want = kv_ref.tree_attention(host(q), *(ref.values(*x) for x in caches), table, lens, bits)
    check_attention(out, lse, *want, "bf16")
    path, n_accept, token = kv.ibp_kv_verify(dev(p, torch.float32), dev(tokens), dev(u, torch.float32), dev(dist, torch.float32),
                                             dev(parents))
    w_path, w_accept, w_token, _ = ref.verify(p, tokens, u, dist, parents)
    assert np.array_equal(host(path), w_path) and np.array_equal(host(n_accept), w_accept) and np.array_equal(host(token), w_token)
    n_draft = dev(np.full(B, T))

    def keep(pair, n, pth, cnt):
        """Moves codes and scales of K and V; the sequences follow once."""
        res = None
        for pages in (*c.k, *c.v):
            res = kv.ibp_kv_accept(pages, t_table, t_lens, t_refs, n, pth, cnt)
        return res

    new = keep(None, n_draft, path, n_accept)
    moved = [kv_ref.accept(x[None], table, lens, refs, [T] * B, w_path, w_accept) for y in caches for x in y]
    caches = [[moved[0][0][0], moved[1][0][0]], [moved[2][0][0], moved[3][0][0]]]
    table, lens, refs = moved[0][1:]
    t_table, t_lens, t_refs = new
    assert np.array_equal(host(t_table), table) and np.array_equal(host(t_lens), lens) and np.array_equal(host(t_refs), refs)
    # one more query for each sequence, its weights, and eviction
    q1 = torch.randn((B, 1, hk * G, D), generator=g, device="cuda").bfloat16()
    out, lse = kv.ibp_kv4_attention(q1, c.k, c.v, t_table, t_lens)
    width = table.shape[1] * page
    was = rng.random((B, width)).astype(np.float32)
    weights = kv.ibp_kv_weigh(q1, c.k, t_table, t_lens, lse, dev(was, torch.float32), decay=0.5)
    want, top = ref.weigh(host(q1), ref.values(*caches[0]), table, lens, host(lse), was, decay=0.5)
    check_weigh(weights, want, top, host(lse), hk * G, was, 0.5)
    e = kv.ibp_kv_evict(weights, t_lens, budget, keep_first=2, keep_last=10)
    w = ref.evict(host(weights), lens, budget, 2, 10)
    assert all(np.array_equal(host(x), y) for x, y in zip(e, w))
    new = keep(None, e[1], e[0], e[2])
    moved = [kv_ref.accept(x[None], table, lens, refs, w[1], w[0], w[2]) for y in caches for x in y]
    caches = [[moved[0][0][0], moved[1][0][0]], [moved[2][0][0], moved[3][0][0]]]
    table, lens, refs = moved[0][1:]
    assert all(np.array_equal(host(x), y) for x, y in zip(new, (table, lens, refs)))
    assert (lens <= budget).all() and (lens == budget).any()
    out, lse = kv.ibp_kv4_attention(q1, c.k, c.v, new[0], new[1])
    check_attention(out, lse, *kv_ref.tree_attention(host(q1), *(ref.values(*x) for x in caches), table, lens), "bf16")


# ---------------------------------------------------------------------------
# Streams, graphs, threads, status


class Step:
    """Every call once, with inputs of its own."""

    def __init__(self, seed=30):
        self.c = Cache([900, 300, 70], 3, 2, 2, 16, 64, seed=seed)
        self.wide = Cache([400, 390] * 3, 40, 4, 4, 64, 64, seed=seed + 1)
        g = gen(seed)
        self.kv = [torch.randn((3, 3, 2, 64), generator=g, device="cuda").bfloat16() for _ in range(2)]
        p, tokens, u, q, parents = draft(5, 6, 20000, True, seed)
        self.v = [dev(p, torch.float32), dev(tokens), dev(u, torch.float32), dev(q, torch.float32), dev(parents)]
        self.w = torch.rand((3, 9000), generator=g, device="cuda")
        self.w2 = torch.rand((6, 500), generator=g, device="cuda")

    def __call__(self, stream=None, **kw):
        """(a call of every kernel)"""
        c, o = self.c, []
        kv.ibp_kv4_store(*self.kv, c.k, c.v, c.table, c.lens, stream=stream, **kw)
        o += kv.ibp_kv4_load(c.k, c.v, c.table, c.lens, 900, n_load=c.lens, stream=stream, **kw)
        out, lse = kv.ibp_kv4_attention(c.q, c.k, c.v, c.table, c.lens, stream=stream, **kw)
        o += [out, lse]
        x = self.wide
        wide, lse_wide = kv.ibp_kv4_attention(x.q, x.k, x.v, x.table, x.lens, stream=stream, **kw)
        o += [wide, lse_wide]
        o += [kv.ibp_kv_weigh(x.q, x.k, x.table, x.lens, lse_wide, self.w2, stream=stream, **kw)]
        o += kv.ibp_kv_verify(*self.v, stream=stream, **kw)
        w = kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, self.w, decay=0.5, stream=stream, **kw)
        o += [w, *kv.ibp_kv_evict(w, c.lens, 64, keep_first=1, keep_last=4, stream=stream, **kw)]
        return o


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


def test_side_streams_and_status_words():
    s = Step()
    want = s()
    torch.cuda.synchronize()
    words = torch.zeros(2, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    one, two = Step(), Step()
    torch.cuda.synchronize()
    for _ in range(3):
        got = one(stream=a, status=words[:1])
        more = two(stream=b.cuda_stream, status=words[1:])
    a.synchronize(), b.synchronize()
    assert same(got, want) and same(more, want) and words.tolist() == [0, 0]


def test_captured_and_replayed():
    kv.ibp_kv_get_status()
    s, t = Step(), Step(40)
    want, other = s(), t()
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in (s, t):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(x())
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            for x in o:
                x.fill_(0)
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    assert same(outs[0], want) and same(outs[1], other)


def test_two_host_threads():
    steps = [Step(), Step(40)]
    want = [s() for s in steps]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(10):
                got = steps[i](stream=stream)
            stream.synchronize()
            if not same(got, want[i]):
                bad.append(i)
        except Exception as e:  # noqa: BLE001 - reported by the main thread
            bad.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_repeats_are_alike():
    """Nothing depends on the order in which threads run."""
    s = Step()
    want = s()
    for _ in range(5):
        assert same(s(), want)


def test_nothing_to_do():
    k4 = cache4(3, 2, 16, 64, "bf16", "hnd", gen(1))
    table, lens = dev(np.zeros((0, 2))), dev(np.zeros(0))
    q = torch.zeros((0, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    kv.ibp_kv4_store(q[:, :, :2], q[:, :, :2], k4, k4, table, lens)
    assert kv.ibp_kv4_load(k4, k4, table, lens, 4)[0].shape == (0, 4, 2, 64)
    out, lse = kv.ibp_kv4_attention(q, k4, k4, table, lens)
    assert out.shape == (0, 1, 4, 64)
    w = torch.zeros((0, 32), device="cuda")
    assert kv.ibp_kv_weigh(q, k4, table, lens, lse, w).shape == (0, 32)
    assert kv.ibp_kv_evict(w, lens, 4)[0].shape == (0, 4)
    z = torch.zeros((0, 3, 50), device="cuda")
    assert kv.ibp_kv_verify(z, dev(np.zeros((0, 2))), torch.zeros((0, 3), device="cuda"))[0].shape == (0, 2)


# ---------------------------------------------------------------------------
# Refusals


def test_refusals():
    g = gen(1)
    k4 = cache4(5, 2, 16, 64, "bf16", "hnd", g)
    table, lens = dev(np.array([[0, 1]])), dev(np.array([20]))
    x = torch.zeros((1, 1, 2, 64), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros((1, 1, 4, 64), dtype=torch.bfloat16, device="cuda")
    attend = lambda q=q, k=k4, v=k4, **kw: kv.ibp_kv4_attention(q, k, v, table, lens, **kw)  # noqa: E731
    lse, w = torch.zeros((1, 1, 4), device="cuda"), torch.zeros((1, 32), device="cuda")
    bad = [
        lambda: kv.ibp_kv4_store(x.half(), x, k4, k4, table, lens),
        lambda: kv.ibp_kv4_store(x[..., :32], x, k4, k4, table, lens),
        lambda: kv.ibp_kv4_store(x, x[:, :, :1], k4, k4, table, lens),
        lambda: kv.ibp_kv4_store(x, x, (k4[0].to(torch.int32), k4[1]), k4, table, lens),
        lambda: kv.ibp_kv4_store(x, x, (k4[0], k4[1].float()), k4, table, lens),
        lambda: kv.ibp_kv4_store(x, x, (k4[0], k4[1][..., :1]), k4, table, lens),
        lambda: kv.ibp_kv4_store(x, x, k4, k4, table.long(), lens),
        lambda: kv.ibp_kv4_store(x, x, k4, k4, table, lens, n_new=lens[:0]),
        lambda: kv.ibp_kv4_load(k4, k4, table, lens, 2, k=x),
        lambda: attend(q.half()), lambda: attend(q[..., :32]), lambda: attend(q.cpu()),
        lambda: attend(v=(k4[0], k4[1].half())),
        lambda: attend(mask=lens), lambda: attend(out=q.float()), lambda: attend(lse=lse[0]),
        lambda: kv.ibp_kv_weigh(q, k4, table, lens, lse[0], w), lambda: kv.ibp_kv_weigh(q, k4, table, lens, lse, w[0]),
        lambda: kv.ibp_kv_weigh(q, k4, table, lens, lse, w.double()),
        lambda: kv.ibp_kv_evict(w, lens, 4, keep_first=3, keep_last=2), lambda: kv.ibp_kv_evict(w, lens, 0),
        lambda: kv.ibp_kv_evict(w, lens, 4, keep_first=-1), lambda: kv.ibp_kv_evict(w, lens.repeat(2), 4),
    ]
    p, t, u = torch.zeros((2, 3, 9), device="cuda"), dev(np.zeros((2, 2))), torch.zeros((2, 3), device="cuda")
    bad += [lambda: kv.ibp_kv_verify(p[:, :2], t, u), lambda: kv.ibp_kv_verify(p.half(), t, u),
            lambda: kv.ibp_kv_verify(p, t, u[:, :2]), lambda: kv.ibp_kv_verify(p, t.long(), u),
            lambda: kv.ibp_kv_verify(p, t, u, q=p), lambda: kv.ibp_kv_verify(p, t, u, parents=t[:1]),
            lambda: kv.ibp_kv_verify(p.transpose(1, 2).contiguous().transpose(1, 2), t, u),
            lambda: kv.ibp_kv_verify(p[..., :0], t, u), lambda: kv.ibp_kv_verify(p, t, u, n_draft=t[0, :1])]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    # what the library itself refuses
    odd = torch.empty(5 * 2 * 16 * 32 + 1, dtype=torch.uint8, device="cuda")[1:].view(5, 2, 16, 32)
    d40 = torch.empty((5, 2, 16, 32), dtype=torch.uint8, device="cuda")
    for call in (lambda: attend(k=(odd, k4[1])), lambda: attend(q=torch.zeros((1, 1, 3, 64), dtype=torch.bfloat16, device="cuda")),
                 lambda: attend(q=q[:, :0], lse=None), lambda: attend(scale=float("nan")),
                 lambda: kv.ibp_kv4_attention(q, k4, (d40[:4], k4[1][:4]), table, lens),
                 lambda: kv.ibp_kv4_store(x[:, :0], x[:, :0], k4, k4, table, lens),
                 lambda: kv.ibp_kv_weigh(q, k4, table, lens, lse, w, decay=float("inf")),
                 lambda: kv.ibp_kv4_load(k4, k4, table, lens.cpu(), 1)):
        with pytest.raises(ibp.IbpError):
            call()
    lib = kv._load()
    n = ctypes.c_void_p(w.data_ptr())
    assert lib.ibp_kv_evict(n, 32, lens.data_ptr(), 1, 4, 0, 0, table.data_ptr(), table.data_ptr(), table.data_ptr(), n, None, None) == ibp.IBP_EINVAL
    many = torch.zeros((1, 64, 4, 64), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="workspace"):
        c = Cache([9000] * 40, 1, 2, 2, 64, 64)
        c.attend(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert many.numel()


def test_a_gradient_is_an_error():
    c = Cache([40], 1, 1, 1, 16, 64)
    c.q.requires_grad_()
    out, lse = c.attend()
    with pytest.raises(RuntimeError, match="no backward"):
        out.sum().backward()
    w = torch.ones((1, 50), device="cuda")
    got = kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse.detach(), w)
    with torch.no_grad():
        assert torch.equal(got, kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, w))
    with pytest.raises(RuntimeError, match="no backward"):
        got.sum().backward()
    w.requires_grad_()
    with pytest.raises(RuntimeError, match="no backward"):
        kv.ibp_kv_evict(w, c.lens, 10)[3].sum().backward()
    with pytest.raises(ValueError, match="in place"):
        kv.ibp_kv_weigh(c.q.detach(), c.k, c.table, c.lens, lse.detach(), w, inplace=True)
    scales = c.k[1].detach().requires_grad_()
    with pytest.raises(RuntimeError, match="no backward"):
        kv.ibp_kv4_load((c.k[0], scales), c.v, c.table, c.lens, 4)[0].sum().backward()


@pytest.mark.parametrize("T,hk,G", [(40, 8, 2), (300, 4, 1), (300, 4, 2)])
def test_waits_that_run_out(T, hk, G):
    """Every wait of the tensor-core kernels gives up: the status says so, and the next call is whole."""
    c = Cache([300, 310, 333], T, hk, G, 16, 64, seed=5)
    want = c.attend()
    torch.cuda.synchronize()
    before = kv.ibp_kv_set_wait_limit(0)
    try:
        c.attend()
        torch.cuda.synchronize()
    finally:
        kv.ibp_kv_set_wait_limit(before)
    err(ibp.IBP_ETIMEOUT)
    assert same(c.attend(), want)


def test_weighing_waits_that_run_out():
    c = Cache([300, 310, 333], 40, 3, 2, 16, 64, seed=5)
    _, lse = c.attend()
    w = torch.ones((3, 400), device="cuda")
    want = kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, w)
    torch.cuda.synchronize()
    before = kv.ibp_kv_set_wait_limit(0)
    try:
        kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, w)
        torch.cuda.synchronize()
    finally:
        kv.ibp_kv_set_wait_limit(before)
    err(ibp.IBP_ETIMEOUT)
    assert torch.equal(kv.ibp_kv_weigh(c.q, c.k, c.table, c.lens, lse, w), want)
