"""Oracle of the caches in 4 bits, the verification of drafted tokens and the
eviction of cached ones: plain loops over numpy arrays, softmax and sums in 64 bits or
in whole numbers.  Shares no code with the CUDA path.

Codes are uint8 arrays [n_pages, heads, page_tokens, dim / 2], scales float arrays
[n_pages, heads, page_tokens, dim / 32].  Functions return new arrays.
"""

import numpy as np

from . import kv_ref

GROUP = 32


# ---------------------------------------------------------------------------
# 4 bits


def scale_of(a, f16):
    """a / 7 to 5 significant bits, ties to even, as the type holds it."""
    part, power = np.frexp(np.float64(a) / 7.0)
    s = np.ldexp(np.rint(part * 32.0) / 32.0, power)
    if f16:
        return np.float64(np.float16(s))
    return np.float64(0.0) if s < 2.0**-100 else min(s, 2.0**121)


def quantise(x, f16):
    """(codes as whole numbers of the dims' shape, scales) of x [..., dim]."""
    x = np.asarray(x, np.float64)
    g = x.reshape(-1, GROUP)
    codes, scales = np.full(g.shape, 8, np.int64), np.zeros(len(g))
    for i, row in enumerate(g):
        if not np.isfinite(row).all():
            scales[i] = np.nan
            continue
        scales[i] = scale_of(np.abs(row).max(), f16)
        if scales[i] > 0:
            codes[i] = 8 + np.clip(np.rint(row / scales[i]), -7, 7)
    return codes.reshape(x.shape), scales.reshape(*x.shape[:-1], -1)


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def values(codes, scales):
    """[..., dim] of packed codes [..., dim / 2] and scales [..., dim / 32]."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).astype(np.float64) - 8
    with np.errstate(invalid="ignore"):
        return c * np.repeat(scales.astype(np.float64), GROUP, -1)


def rows(lens, n_rows, T, table, page, n_pages):
    """(sequence, row, page id, slot) of every row with a position and a page."""
    for b in range(len(lens)):
        n = T if n_rows is None else min(max(int(n_rows[b]), 0), T)
        for t in range(n):
            pos = int(lens[b]) - n + t
            if pos >= 0 and 0 <= table[b, pos // page] < n_pages:
                yield b, t, int(table[b, pos // page]), pos % page


def store(x, codes, scales, table, lens, n_new, f16):
    codes, scales = codes.copy(), scales.copy()
    for b, t, pg, slot in rows(lens, n_new, x.shape[1], table, codes.shape[2], codes.shape[0]):
        c, s = quantise(x[b, t], f16)
        codes[pg, :, slot], scales[pg, :, slot] = pack(c), s
    return codes, scales


def load(codes, scales, table, lens, T, n_load):
    out = np.zeros((len(lens), T, codes.shape[1], codes.shape[3] * 2))
    for b, t, pg, slot in rows(lens, n_load, T, table, codes.shape[2], codes.shape[0]):
        out[b, t] = values(codes[pg, :, slot], scales[pg, :, slot])
    return out


# ---------------------------------------------------------------------------
# Drafted tokens


def verify(p, tokens, u, q=None, parents=None, n_draft=None):
    """(path, n_accept, token, whether anything was out of range)"""
    f32 = np.float32
    B, T = tokens.shape
    V = p.shape[2]

    def clean(row):
        return np.clip(np.where(np.isnan(row), f32(0), row), f32(0), f32(1)).astype(f32)

    def whole(w):
        return [int(x) for x in np.rint(w.astype(np.float64) * 2.0**44)]

    path, count, token, bad = np.full((B, T), -1, np.int32), np.zeros(B, np.int32), np.full(B, -1, np.int32), False
    for b in range(B):
        n = T if n_draft is None else int(n_draft[b])
        bad |= not 0 <= n <= T
        n = min(max(n, 0), T)
        node, left = -1, clean(p[b, 0])
        draw = left
        for t in range(n):
            x, parent = int(tokens[b, t]), t - 1 if parents is None else int(parents[b, t])
            if not 0 <= x < V or not -1 <= parent < t:
                bad = True
                continue
            if parent != node:
                continue
            if q is None:
                drawn = np.zeros(V, f32)
                drawn[x] = 1
            else:
                drawn = clean(q[b, parent + 1])
            if float(u[b, t]) * float(drawn[x]) < float(left[x]):
                path[b, count[b]] = node = t
                count[b] += 1
                left = draw = clean(p[b, t + 1])
                continue
            rest = np.maximum(left - drawn, f32(0))
            Z = sum(whole(rest))
            if Z > 0:
                draw, left = rest, rest * f32(2.0**44 / float(Z))
        weight = whole(draw)
        total = sum(weight)
        if total == 0:
            bad = True
            continue
        r = float(u[b, T])
        aim = 0 if not r > 0 else min(int(min(r * float(total), 2.0**62)), total - 1)
        run = 0
        for i, w in enumerate(weight):
            run += w
            if run > aim:
                token[b] = i
                break
    return path, count, token, bad


# ---------------------------------------------------------------------------
# Eviction


def weigh(q, keys, table, lens, lse, w, mask=None, n_draft=None, scale=None, decay=1.0):
    """(weights, their sums of magnitudes, largest |q k| sum) with keys [n_pages, heads, tokens, dim]."""
    B, T, H, D = q.shape
    G = H // keys.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, top = w.astype(np.float64).copy(), 0.0
    for b in range(B):
        n = T if n_draft is None else min(max(int(n_draft[b]), 0), T)
        length, ctx = int(lens[b]), int(lens[b]) - n
        for j in range(min(length, w.shape[1])):
            out[b, j] = decay * np.float64(w[b, j]) if j < ctx else 0.0
        spots = list(range(min(length, w.shape[1])))
        for h in range(keys.shape[1]):
            k = kv_ref.rows_of(keys, table[b], spots, h)
            for t in range(n):
                sees = [j for j in spots if j < ctx or kv_ref.tree_sees(mask, b, t, j - ctx)]
                for g in range(h * G, h * G + G):
                    if lse[b, t, g] == -np.inf or not sees:
                        continue
                    qq = q[b, t, g].astype(np.float64)
                    out[b, sees] += np.exp(k[sees] @ qq * scale - np.float64(lse[b, t, g]))
                    top = max(top, float((np.abs(k[sees]) @ np.abs(qq)).max() * abs(scale)))
    return out, top


def evict(w, lens, budget, keep_first, keep_last):
    """(path, n_draft, n_keep, weights)"""
    B, width = w.shape
    path, n_draft, n_keep = np.full((B, budget), -1, np.int32), np.zeros(B, np.int32), np.zeros(B, np.int32)
    out = np.zeros_like(w)
    for b in range(B):
        n = int(lens[b])
        if not 0 <= n <= width:  # left alone
            out[b] = w[b] if n > width else 0
            continue
        kept = list(range(n))
        if n > budget:
            forced = [i for i in kept if i < keep_first or i >= n - keep_last]
            rest = [i for i in kept if keep_first <= i < n - keep_last]
            rest.sort(key=lambda i: (np.isnan(w[b, i]), -w[b, i] if not np.isnan(w[b, i]) else 0, i))
            kept = sorted(forced + rest[: budget - len(forced)])
            path[b], n_draft[b], n_keep[b] = kept, n, budget
        out[b, : len(kept)] = w[b, kept]
    return path, n_draft, n_keep, out
