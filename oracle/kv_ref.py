"""Oracle of the paged key/value cache operators: plain loops over numpy arrays,
sums and softmax in 64 bits.  Shares no code with the CUDA path.

Keys and values are float arrays [n_pages, heads, page_tokens, dim]; tables,
lengths and reference counts are integer arrays.  Functions return new arrays.
"""

import numpy as np


def held(n, page):
    return -(-n // page)


# ---------------------------------------------------------------------------
# Pages


def fork(table, lens, refs, parents, page):
    """(table, lens, refs, moves, out_of_pages)"""
    refs = refs.copy()
    n, width = len(parents), table.shape[1]
    out = np.full((n, width), -1, np.int32)
    new_lens = np.zeros(n, np.int32)
    for r in range(len(lens)):
        for p in range(held(lens[r], page)):
            refs[table[r, p]] -= 1
    owner = {}
    wants = []
    for i, par in enumerate(parents):
        new_lens[i] = lens[par]
        for p in range(held(lens[par], page)):
            pg = int(table[par, p])
            if p == lens[par] // page and owner.setdefault(pg, i) != i:
                wants.append(i)
                continue
            out[i, p] = pg
            refs[pg] += 1
    moves, short = [], False
    free = [p for p in range(len(refs)) if refs[p] == 0]
    for i in wants:
        full, part = divmod(int(new_lens[i]), page)
        if not free:
            new_lens[i] = full * page
            short = True
            continue
        to = free.pop(0)
        out[i, full] = to
        refs[to] = 1
        moves.append((int(table[parents[i], full]), to, part))
    return out, new_lens, refs, moves, short


def free(table, lens, refs, seqs, page):
    table, lens, refs = table.copy(), lens.copy(), refs.copy()
    for s in seqs:
        for p in range(held(lens[s], page)):
            refs[table[s, p]] -= 1
        if lens[s]:
            table[s] = -1
        lens[s] = 0
    return table, lens, refs


def compact(table, refs, page):
    """(table, refs, moves)"""
    live = [p for p in range(len(refs)) if refs[p] > 0]
    n = len(live)
    holes = [p for p in range(n) if refs[p] <= 0]
    movers = [p for p in live if p >= n]
    to = dict(zip(movers, holes))
    out = np.array([[to.get(int(p), int(p)) if p >= 0 else -1 for p in row] for row in table], np.int32)
    new = refs.copy()
    for a, b in to.items():
        new[b], new[a] = refs[a], 0
    return out.reshape(table.shape), new, [(a, b, page) for a, b in to.items()]


def copy(pool, moves):
    """pool [..., n_pages, heads, tokens, dim]"""
    new = pool.copy()
    for a, b, n in moves:
        new[..., b, :, :n, :] = pool[..., a, :, :n, :]
    return new


def accept(pool, table, lens, refs, n_draft, path, n_accept):
    """(pool, table, lens, refs)"""
    page = pool.shape[-2]
    new, table, lens, refs = pool.copy(), table.copy(), lens.copy(), refs.copy()
    for b in range(len(lens)):
        ctx = int(lens[b] - n_draft[b])
        for j in range(n_accept[b]):
            s, d = ctx + int(path[b, j]), ctx + j
            new[..., table[b, d // page], :, d % page, :] = pool[..., table[b, s // page], :, s % page, :]
        was, lens[b] = held(lens[b], page), ctx + n_accept[b]
        now = held(lens[b], page)
        for p in range(now, was):
            refs[table[b, p]] -= 1
        table[b, now:] = -1
    return new, table, lens, refs


# ---------------------------------------------------------------------------
# Attention


def attend(q, keys, vals, scale):
    """One query over the keys it sees: (out, lse, mean of |v|, largest sum of
    |q k|), the last two for error bounds."""
    if len(keys) == 0:
        return np.zeros(len(q)), -np.inf, np.zeros(len(q)), 0.0
    s = (keys @ q) * scale
    m = s.max()
    p = np.exp(s - m)
    total = p.sum()
    return ((p @ vals) / total, m + np.log(total), (p @ np.abs(vals)) / total,
            float((np.abs(keys) @ np.abs(q)).max() * abs(scale)))


def rows_of(pages, table_row, positions, head):
    """Keys or values of one head at the given positions, as float64; a page id out
    of range reads as zeros."""
    page = pages.shape[2]
    out = np.zeros((len(positions), pages.shape[3]))
    for i, p in enumerate(positions):
        pg = table_row[p // page]
        if 0 <= pg < pages.shape[0]:
            out[i] = pages[pg, head, p % page]
    return out


def tree_sees(mask, b, t, i):
    return i <= t if mask is None else bool((int(mask[b, t, i // 32]) >> (i % 32)) & 1)


def tree_attention(q, k, v, table, lens, mask=None, n_draft=None, scale=None):
    """(out, lse, mean |v|, largest |q k|) in float64, q [n_seqs, T, heads, dim]"""
    B, T, H, D = q.shape
    G = H // k.shape[1]
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, lse, mean, top = np.zeros(q.shape), np.full((B, T, H), -np.inf), np.zeros(q.shape), np.zeros((B, T, H))
    for b in range(B):
        n = T if n_draft is None else int(n_draft[b])
        ctx = int(lens[b]) - n
        for t in range(n):
            spots = list(range(max(ctx, 0))) + [ctx + i for i in range(n) if ctx + i >= 0 and tree_sees(mask, b, t, i)]
            for h in range(k.shape[1]):
                keys, vals = rows_of(k, table[b], spots, h), rows_of(v, table[b], spots, h)
                for g in range(h * G, h * G + G):
                    out[b, t, g], lse[b, t, g], mean[b, t, g], top[b, t, g] = attend(
                        q[b, t, g].astype(np.float64), keys, vals, scale)
    return out, lse, mean, top


def summarize(k, table, lens, codes, scales, first=None):
    """Codes and scales with the touched pages' entries computed anew."""
    page = k.shape[2]
    codes, scales = codes.copy(), scales.copy()
    f32 = np.float32
    for b in range(len(lens)):
        start = 0 if first is None else max(0, int(first[b]))
        for p in range(start // page, held(lens[b], page)):
            if start >= lens[b]:
                break
            keys = k[table[b, p], :, : min(page, lens[b] - p * page)].astype(f32)
            for h in range(k.shape[1]):
                a = np.abs(keys[h]).max()
                at = table[b, p], h
                if not np.isfinite(keys[h]).all():
                    codes[at], scales[at] = 0, np.inf
                elif a < f32(2.0**-100):
                    codes[at], scales[at] = 0, 0
                else:
                    f = f32(f32(1) / a) * f32(127)
                    ends = np.stack([keys[h].min(0), keys[h].max(0)])
                    codes[at] = np.clip(np.rint(ends * f), -127, 127)
                    scales[at] = a * (f32(1) / f32(127))
    return codes, scales


def select(q, codes, scales, table_row, place, page, budget, keep_first, keep_last):
    """Pages one query and kv head attends to; q [group, dim] float32, codes
    [n_pages, 2, dim] and scales [n_pages] of the kv head."""
    near = place // page
    if near + 1 <= budget:
        return list(range(near + 1))
    a = np.abs(q).max()
    c = np.zeros(q.shape, np.int64)
    if np.isfinite(q).all() and a >= np.float32(2.0**-100):
        f = np.float32(np.float32(1) / a) * np.float32(127)
        c = np.clip(np.rint(q.astype(np.float32) * f), -127, 127).astype(np.int64)
    forced = [p for p in range(near + 1) if p < keep_first or p > near - keep_last]
    scored = []
    for p in range(near + 1):
        if p in forced:
            continue
        lo, hi = codes[table_row[p]].astype(np.int64)
        total = int((np.maximum(c, 0) * hi + np.minimum(c, 0) * lo).sum())
        s = scales[table_row[p]]
        scored.append((-(np.float32(total) * s) if np.isfinite(s) else -np.inf, p))
    scored.sort()
    return sorted(forced + [p for _, p in scored[: budget - len(forced)]])


def sparse_attention(q, k, v, table, lens, codes, scales, budget, keep_first, keep_last, n_query=None, scale=None):
    """(out, lse, pages, mean |v|, largest |q k|)"""
    B, T, H, D = q.shape
    hk, page = k.shape[1], k.shape[2]
    G = H // hk
    scale = 1 / np.sqrt(D) if scale is None else scale
    out, lse, mean, top = np.zeros(q.shape), np.full((B, T, H), -np.inf), np.zeros(q.shape), np.zeros((B, T, H))
    pages = np.full((B, T, hk, budget), -1, np.int32)
    for b in range(B):
        n = T if n_query is None else int(n_query[b])
        for t in range(n):
            place = int(lens[b]) - n + t
            if place < 0:
                continue
            for h in range(hk):
                group = q[b, t, h * G : (h + 1) * G]
                picked = select(group, codes[:, h], scales[:, h], table[b], place, page, budget, keep_first, keep_last)
                pages[b, t, h, : len(picked)] = picked
                spots = [p * page + i for p in picked for i in range(page) if p * page + i <= place]
                keys, vals = rows_of(k, table[b], spots, h), rows_of(v, table[b], spots, h)
                for g in range(G):
                    at = b, t, h * G + g
                    out[at], lse[at], mean[at], top[at] = attend(group[g].astype(np.float64), keys, vals, scale)
    return out, lse, pages, mean, top
