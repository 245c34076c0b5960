"""Helpers of the paged cache tests: pools, page tables and error bounds."""

import numpy as np
import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
UNIT = {"bf16": 2.0**-8, "f16": 2.0**-11}  # rounding to nearest of a value of 1


def pool(shape, dtype, layout, gen, fill=None):
    """Pages [..., n_pages, heads, tokens, dim] in one of three memory orders, and
    with padding between pages for the third."""
    *lead, n, h, t, d = shape
    if layout == "hnd":
        x = torch.empty((*lead, n, h, t, d), dtype=dtype, device="cuda")
    elif layout == "nhd":
        x = torch.empty((*lead, n, t, h, d), dtype=dtype, device="cuda").transpose(-2, -3)
    else:  # padded tokens, heads and pages; what lies between is NaN
        x = torch.full((*lead, n, h + 1, t + 1, d + 8), float("nan"), dtype=dtype, device="cuda")
        x = x[..., :h, :t, :d]
    x.normal_(generator=gen) if fill is None else x.fill_(fill)
    return x


def tables(lens, page, n_pages, width, rng):
    """Random disjoint pages for sequences of the given lengths."""
    order = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, np.int32)
    refs = np.zeros(n_pages, np.int32)
    at = 0
    for b, n in enumerate(lens):
        k = -(-n // page)
        table[b, :k] = order[at : at + k]
        refs[order[at : at + k]] = 1
        at += k
    assert at <= n_pages
    return table, refs


def poison(pages, table, lens, value=float("nan")):
    """Sets every token of the pool that no sequence holds."""
    page = pages.shape[2]
    hit = np.ones((pages.shape[0], page), bool)
    for b, n in enumerate(lens):
        for p in range(n):
            if 0 <= table[b, p // page] < pages.shape[0]:
                hit[table[b, p // page], p % page] = False
    m = torch.from_numpy(hit).cuda()[:, None, :, None]
    pages.masked_fill_(m, value)


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.detach().cpu().numpy()


def check_attention(out, lse, want, want_lse, mean, top, dt):
    """Compares with the 64-bit oracle.  Bound per element: the output's own
    rounding (u |out|); the probabilities' rounding to the cache's type (u, or
    2^-25 absolute for small half-precision ones, times the mean of |v|, as a
    sum of at least one); and the scores' error, (dim + 8) 2^-23 of the largest
    sum of |q k| plus 2^-20 for the exponential, twice (numerator and sum)."""
    u, D = UNIT[dt], want.shape[-1]
    eps = (D + 8) * 2.0**-23 * top + 2.0**-20
    tol = u * np.abs(want) * 1.01 + (u + 2 * eps[..., None]) * mean * 1.02 + (2.0**-24 * 64 if dt == "f16" else 0)
    got, got_lse = host(out).astype(np.float64), host(lse).astype(np.float64)
    assert np.isfinite(got).all()
    bad = np.abs(got - want) - tol
    assert (bad <= 0).all(), f"out off by {bad.max():.3g} beyond the bound at {np.unravel_index(bad.argmax(), bad.shape)}"
    empty = want_lse == -np.inf
    assert (got_lse[empty] == -np.inf).all() and (got[empty] == 0).all()
    off = np.abs(got_lse[~empty] - want_lse[~empty]) - (eps[~empty] + 2.0**-20 * (1 + np.abs(want_lse[~empty])))
    assert off.size == 0 or (off <= 0).all(), f"lse off by {off.max():.3g} beyond the bound"
