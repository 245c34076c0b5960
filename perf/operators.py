"""Cases of the paged key/value cache operators: what is timed and compared.

Five kinds of pass, each as a serving program makes it:

fork       a beam step: the next batch of sequences from its parents (shared
           pages, copies of partly filled last pages), then the page copies
retire     finished sequences are freed, the pool is compacted to its front,
           then the page copies
accept     the accepted drafted tokens of each sequence move to the front of
           its draft, and the pages behind them are freed
summarize  8-bit bounds of the keys of the pages that new tokens touched
tree       attention of a tree of drafted tokens over the paged cache
sparse     selection of pages by the cheap score of their bounds for each
           query, and attention over the selected pages

`own = False` computes a pass by elementary torch operations in 32 bits,
`own = True` by the framework's entry points (host_transfer_gb300.kv).
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------
# Cases


def listed():
    return [
        # a beam step of a small two-layer draft model: latency counts
        dict(name="fork_small", kind="fork", pools=4, heads=8, page=16, dim=64, dtype="bf16", layout="hnd",
             seqs=4, length=75, pages=48),
        # a beam step of 32 layers of 32 heads x 128 (the LLM configuration's cache), half of the last pages copied
        dict(name="fork_llm", kind="fork", pools=64, heads=32, page=64, dim=128, dtype="bf16", layout="hnd",
             seqs=24, length=300, pages=128),
        # a batch's end: a third of the sequences leave, the live pages move to the pool's front
        dict(name="retire_llm", kind="retire", pools=64, heads=32, page=64, dim=128, dtype="f16", layout="hnd",
             seqs=24, length=300, pages=160),
        # the end of a verification step, tokens-first page layout, 16-token pages
        dict(name="accept_batch", kind="accept", pools=64, heads=32, page=16, dim=128, dtype="bf16", layout="nhd",
             seqs=61, length=37, draft=24, pages=256),
        # a decode step: only the last page of each sequence gets new bounds
        dict(name="summarize_step", kind="summarize", heads=8, page=64, dim=128, dtype="bf16", layout="hnd",
             seqs=16, length=4096, fresh=1),
        # after a long prefill: bounds of every page, odd lengths
        dict(name="summarize_prefill", kind="summarize", heads=8, page=64, dim=128, dtype="f16", layout="hnd",
             seqs=16, length=32749, fresh=32749),
        # one sequence, one token: the latency of a decode step
        dict(name="tree_token", kind="tree", seqs=1, draft=1, qheads=32, heads=8, page=16, dim=128, dtype="bf16",
             layout="hnd", length=777),
        # the LLM configuration's cache (32 heads x 128, 4096 tokens), 13 drafted tokens, a ragged batch
        dict(name="tree_llm", kind="tree", seqs=8, draft=13, qheads=32, heads=32, page=64, dim=128, dtype="bf16",
             layout="hnd", length=4096),
        # wide trees over long caches with grouped heads: the tensor cores' work and the cache's bytes both count
        dict(name="tree_wide", kind="tree", seqs=16, draft=64, qheads=64, heads=8, page=64, dim=128, dtype="f16",
             layout="hnd", length=32768),
        # one sequence, one token, small pages: the latency of a sparse decode step
        dict(name="sparse_token", kind="sparse", seqs=1, draft=1, qheads=32, heads=8, page=16, dim=128,
             dtype="bf16", layout="hnd", length=8191, budget=32, first=1, last=2),
        # a decode batch over long caches: one page in eight or fewer is read
        dict(name="sparse_batch", kind="sparse", seqs=32, draft=1, qheads=32, heads=8, page=64, dim=128,
             dtype="bf16", layout="hnd", length=65536, budget=64, first=1, last=2),
        # a chunk of a prompt, each token with its own pages; half-precision, 64-wide heads, tokens-first layout
        dict(name="sparse_chunk", kind="sparse", seqs=2, draft=511, qheads=32, heads=4, page=32, dim=64,
             dtype="f16", layout="nhd", length=16384, budget=24, first=1, last=1),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["fork", "retire", "accept", "summarize", "tree", "tree", "sparse", "sparse"])
    c = dict(kind=kind, dtype=rng.choice(["bf16", "f16"]), layout=rng.choice(["hnd", "nhd"]),
             page=rng.choice([16, 16, 24, 32, 64, 128]), dim=rng.choice([64, 80, 128, 128]))
    if kind in ("fork", "retire", "accept"):
        c["heads"] = rng.choice([1, 2, 8, 32])
        c["pools"] = 2 * _spread(rng, 1, 32)
        c["seqs"] = _spread(rng, 1, 48)
        if kind == "accept":
            c["draft"] = _spread(rng, 1, 40)
            c["length"] = c["draft"] + _spread(rng, 1, 200)
        else:
            c["length"] = _spread(rng, 1, 400)
        need = 2 * c["seqs"] * (c["length"] // c["page"] + 1) + 3
        c["pages"] = need
        while c["pools"] > 2 and 2 * c["pools"] * c["heads"] * c["page"] * c["dim"] * need > 4 << 30:
            c["pools"] -= 2
        while c["heads"] > 1 and 2 * c["pools"] * c["heads"] * c["page"] * c["dim"] * need > 4 << 30:
            c["heads"] //= 2
        return c
    c["heads"] = rng.choice([1, 2, 4, 8, 32])
    c["seqs"] = _spread(rng, 1, 32)
    c["length"] = _spread(rng, 1, 32768)
    if kind == "summarize":
        c["fresh"] = _spread(rng, 1, c["length"])
    else:
        c["qheads"] = c["heads"] * rng.choice([g for g in (1, 2, 4, 7, 8, 16) if g * c["heads"] <= 64])
        c["draft"] = rng.choice([1, _spread(rng, 1, 64)])
        c["length"] = max(c["length"], c["draft"])
        if kind == "sparse":
            c["first"], c["last"] = rng.choice([0, 1, 2]), rng.choice([1, 1, 2, 3])
            c["budget"] = c["first"] + c["last"] + _spread(rng, 1, 60)
            if c["draft"] == 1:
                c["draft"] = rng.choice([1, 1, _spread(rng, 2, 256)])
            while c["seqs"] > 1 and c["seqs"] * c["draft"] * c["qheads"] * c["budget"] * c["page"] > 1 << 28:
                c["seqs"] //= 2
            c["length"] = max(c["length"], c["draft"])
    while c["seqs"] > 1 and c["seqs"] * c["heads"] * c["length"] > 16 * 8 * 32768:
        c["seqs"] //= 2
    return c


def _lens(c):
    """Lengths of a ragged batch: the first sequence is the longest, the others at least three tenths of it."""
    low = c.get("draft", 1)
    return [max(low, c["length"] - int(0.7 * c["length"] * ((i * 0.6180339887) % 1.0))) for i in range(c["seqs"])]


# --------------------------------------------------------------------------
# Inputs


def _pool(shape, layout, dtype, gen):
    """Pages [..., pages, heads, tokens, dim] whose memory is in that order, or tokens before heads."""
    *outer, heads, page, dim = shape
    stored = (*outer, heads, page, dim) if layout == "hnd" else (*outer, page, heads, dim)
    x = torch.empty(stored, dtype=dtype, device="cuda").normal_(generator=gen)
    return x if layout == "hnd" else x.transpose(-2, -3)


def _sequences(c, lens, n_pages, gen, extra=0):
    """Page table, lengths and reference counts; the pages are drawn without order from the pool."""
    need = [-(-n // c["page"]) for n in lens]
    width = max(need) + extra
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    lens_t = torch.tensor(lens, dtype=torch.int32, device="cuda")
    need_t = torch.tensor(need, device="cuda")
    at = torch.arange(width, device="cuda")
    base = torch.cumsum(need_t, 0) - need_t
    held = at < need_t[:, None]
    table = torch.where(held, order[(base[:, None] + at).clamp(max=n_pages - 1)], -1).to(torch.int32)
    refs = torch.zeros(n_pages + 1, dtype=torch.int32, device="cuda")
    refs.scatter_add_(0, torch.where(held, table, n_pages).reshape(-1).long(),
                      torch.ones(table.numel(), dtype=torch.int32, device="cuda"))
    return table.contiguous(), lens_t, refs[:n_pages].contiguous()


def _bounds(k, valid):
    """Codes and scales of key bounds; k [..., tokens, dim] in 32 bits, valid [..., tokens]."""
    seen = valid[..., None]
    amax = torch.where(seen, k.abs(), 0.0).amax(-1).amax(-1)
    bad = (~torch.isfinite(k) & seen).any(-1).any(-1)
    fine = ~bad & (amax >= 2.0**-100)
    inv = torch.where(fine, 127.0 / torch.where(fine, amax, 1.0), 0.0)
    lo = torch.where(seen, k, math.inf).amin(-2)
    hi = torch.where(seen, k, -math.inf).amax(-2)
    code = torch.round(torch.where(fine[..., None, None], torch.stack([lo, hi], -2), 0.0) * inv[..., None, None])
    scale = torch.where(bad, math.inf, torch.where(fine, amax / 127.0, 0.0))
    return code.clamp(-127, 127).to(torch.int8), scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 1)
    dt = DT[c["dtype"]]
    lens = _lens(c)
    if c["kind"] in ("fork", "retire", "accept"):
        table, lens_t, refs = _sequences(c, lens, c["pages"], gen, extra=1)
        s = dict(case=c, table=table, lens=lens_t, refs=refs)
        s["pool"] = _pool((c["pools"], c["pages"], c["heads"], c["page"], c["dim"]), c["layout"], dt, gen)
        n = c["seqs"]
        if c["kind"] == "fork":
            s["parents"] = torch.randint(0, n, (n,), generator=gen, device="cuda", dtype=torch.int32)
        elif c["kind"] == "retire":
            gone = torch.randperm(n, generator=gen, device="cuda")[: max(1, n // 3)]
            s["seqs"] = gone.sort().values.to(torch.int32)
        else:
            # the best first candidate is accepted, then deeper nodes, which come behind the first level
            T = c["draft"]
            depth = max(1, min(8, T // 4))
            s["n_draft"] = torch.full((n,), T, dtype=torch.int32, device="cuda")
            s["n_accept"] = torch.randint(0, depth + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
            at = torch.rand(n, max(T - depth, 1), generator=gen, device="cuda").argsort(1)[:, : depth - 1]
            path = torch.cat([torch.zeros(n, 1, device="cuda"), depth + at.sort(1).values], 1)
            s["path"] = path.to(torch.int32).contiguous()
        return s
    need = sum(-(-n // c["page"]) for n in lens)
    n_pages = need + 5
    table, lens_t, _ = _sequences(c, lens, n_pages, gen)
    # keys of a page share a direction, as those of neighbouring tokens do; scales differ from head to head
    k = _pool((n_pages, c["heads"], c["page"], c["dim"]), c["layout"], dt, gen)
    k += torch.randn(n_pages, c["heads"], 1, c["dim"], generator=gen, device="cuda").to(dt)
    k *= torch.empty(c["heads"], 1, 1, device="cuda").uniform_(0.5, 2.0, generator=gen).to(dt)
    s = dict(case=c, table=table, lens=lens_t, k=k)
    if c["kind"] == "summarize":
        s["codes"] = torch.zeros(n_pages, c["heads"], 2, c["dim"], dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(n_pages, c["heads"], device="cuda")
        s["first"] = (lens_t - c["fresh"]).clamp(min=0)
        return s
    T = c["draft"]
    s["v"] = _pool((n_pages, c["heads"], c["page"], c["dim"]), c["layout"], dt, gen)
    s["q"] = torch.randn(c["seqs"], T, c["qheads"], c["dim"], generator=gen, device="cuda").to(dt)
    if c["kind"] == "tree":
        # a random tree: each node's parent is an earlier node of the last eight, or the context's last token
        at = torch.arange(T, device="cuda")
        back = torch.randint(1, 9, (c["seqs"], T), generator=gen, device="cuda")
        reach = torch.eye(T, dtype=torch.bool, device="cuda").repeat(c["seqs"], 1, 1)
        reach |= (at[None, :, None] - back[:, :, None]) == at[None, None, :]
        for _ in range(max(1, T.bit_length())):
            reach = torch.bmm(reach.float(), reach.float()) > 0
        bits = torch.nn.functional.pad(reach, (0, -T % 32)).reshape(c["seqs"], T, -1, 32).long()
        words = (bits << torch.arange(32, device="cuda")).sum(-1)
        s["mask"] = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    else:
        valid = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
        at = torch.arange(table.shape[1], device="cuda") * c["page"]
        left = (lens_t[:, None] - at).clamp(0, c["page"]).to(torch.int32)
        held = left > 0
        valid[table[held].long()] = left[held]
        seen = torch.arange(c["page"], device="cuda") < valid[:, None, None]
        parts = [_bounds(a.float(), b.expand(a.shape[:-1])) for a, b in zip(k.split(4096), seen.split(4096))]
        s["codes"] = torch.cat([p[0] for p in parts]).contiguous()
        s["scales"] = torch.cat([p[1] for p in parts]).contiguous()
    return s


# --------------------------------------------------------------------------
# One pass


def run(state):
    return (_own if own else _plain)[state["case"]["kind"]](state)


def _own_fork(s):
    from host_transfer_gb300 import kv

    table, lens, refs, moves, count = kv.ibp_kv_fork(s["table"], s["lens"], s["refs"], s["parents"],
                                                     s["case"]["page"])
    kv.ibp_kv_copy(s["pool"], moves, count)
    return dict(table=table, lens=lens, refs=refs, moves=moves, count=count, pool=s["pool"])


def _own_retire(s):
    from host_transfer_gb300 import kv

    table, lens, refs = kv.ibp_kv_free(s["table"], s["lens"], s["refs"], s["seqs"], s["case"]["page"])
    table, refs, moves, count = kv.ibp_kv_compact(table, refs, s["case"]["page"])
    kv.ibp_kv_copy(s["pool"], moves, count)
    return dict(table=table, lens=lens, refs=refs, moves=moves, count=count, pool=s["pool"])


def _own_accept(s):
    from host_transfer_gb300 import kv

    table, lens, refs = kv.ibp_kv_accept(s["pool"], s["table"], s["lens"], s["refs"], s["n_draft"], s["path"],
                                         s["n_accept"])
    return dict(table=table, lens=lens, refs=refs, pool=s["pool"])


def _own_summarize(s):
    from host_transfer_gb300 import kv

    kv.ibp_kv_summarize(s["k"], s["table"], s["lens"], s["codes"], s["scales"], first=s["first"])
    return dict(bounds=s["codes"] * s["scales"][..., None, None], scales=s["scales"])


def _own_tree(s):
    from host_transfer_gb300 import kv

    out, lse = kv.ibp_tree_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], mask=s["mask"])
    return dict(out=out, lse=lse)


def _own_sparse(s):
    from host_transfer_gb300 import kv

    c = s["case"]
    out, lse, pages = kv.ibp_sparse_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], s["codes"],
                                              s["scales"], c["budget"], keep_first=c["first"],
                                              keep_last=c["last"])
    return dict(out=out, lse=lse, pages=pages)


_own = dict(fork=_own_fork, retire=_own_retire, accept=_own_accept, summarize=_own_summarize, tree=_own_tree,
            sparse=_own_sparse)


def _count_pages(pages, held, n_pages):
    """How often each page is held: pages and held alike in shape."""
    at = torch.where(held, pages, n_pages).reshape(-1).long()
    one = torch.ones_like(at, dtype=torch.int32)
    return torch.zeros(n_pages + 1, dtype=torch.int32, device=at.device).scatter_add_(0, at, one)[:n_pages]


def _move_pages(pool, src, dst, tokens):
    """Copies the first tokens of pages src onto pages dst in every pool."""
    page = torch.arange(pool.shape[3], device=pool.device)
    seen = (page < tokens[:, None])[None, :, None, :, None]
    pool[:, dst] = torch.where(seen, pool[:, src], pool[:, dst])


def _plain_fork(s):
    page, n_pages = s["case"]["page"], s["refs"].numel()
    par = s["parents"].long()
    at = torch.arange(s["table"].shape[1], device=par.device)
    table, lens = s["table"][par], s["lens"][par]
    rows = torch.arange(par.numel(), device=par.device)
    held_in = at < ((s["lens"] + page - 1) // page)[:, None]
    full, part = (lens // page).long(), lens % page
    tail = table.gather(1, full.clamp(max=at.numel() - 1)[:, None])[:, 0].long()
    key = torch.where(part > 0, tail, n_pages)
    owner = torch.full((n_pages + 1,), par.numel(), device=par.device).scatter_reduce_(0, key, rows, "amin")
    need = (part > 0) & (owner[key] != rows)
    held = at < ((lens + page - 1) // page)[:, None]
    shared = held & ~(need[:, None] & (at == full[:, None]))
    refs = s["refs"] - _count_pages(s["table"], held_in, n_pages) + _count_pages(table, shared, n_pages)
    free = torch.sort((refs != 0).int(), stable=True).indices
    rank = torch.cumsum(need, 0) - 1
    got = need & (rank < (refs == 0).sum())
    fresh = free[rank.clamp(0, n_pages - 1)]
    table = torch.where(held & (got[:, None] | shared), table, -1)
    table = torch.where(got[:, None] & (at == full[:, None]), fresh[:, None].to(torch.int32), table)
    lens = torch.where(need & ~got, lens - part, lens)
    refs = refs + _count_pages(fresh, got, n_pages)
    rows = got.nonzero()[:, 0]
    moves = torch.full((par.numel(), 3), -1, dtype=torch.int32, device=par.device)
    moves[: rows.numel()] = torch.stack([tail[rows], fresh[rows], part[rows]], 1).to(torch.int32)
    _move_pages(s["pool"], tail[rows], fresh[rows], part[rows])
    count = got.sum().to(torch.int32).reshape(1)
    return dict(table=table, lens=lens, refs=refs, moves=moves, count=count, pool=s["pool"])


def _plain_retire(s):
    page, n_pages = s["case"]["page"], s["refs"].numel()
    at = torch.arange(s["table"].shape[1], device="cuda")
    gone = torch.zeros_like(s["lens"], dtype=torch.bool).index_fill_(0, s["seqs"].long(), True)
    held = at < ((s["lens"] + page - 1) // page)[:, None]
    refs = s["refs"] - _count_pages(s["table"], held & gone[:, None], n_pages)
    table = torch.where(gone[:, None], -1, s["table"])
    lens = torch.where(gone, 0, s["lens"])
    live = refs > 0
    n_live = live.sum()
    ids = torch.arange(n_pages, device="cuda")
    dst, src = (~live & (ids < n_live)).nonzero()[:, 0], (live & (ids >= n_live)).nonzero()[:, 0]
    to = ids.to(torch.int32).index_copy(0, src, dst.to(torch.int32))
    table = torch.where(table >= 0, to[table.clamp(min=0).long()], -1)
    refs = refs.index_copy(0, dst, refs[src]).index_fill(0, src, 0)
    moves = torch.full((n_pages, 3), -1, dtype=torch.int32, device="cuda")
    tokens = torch.full_like(src, page)
    moves[: src.numel()] = torch.stack([src, dst, tokens], 1).to(torch.int32)
    _move_pages(s["pool"], src, dst, tokens)
    count = torch.tensor([src.numel()], dtype=torch.int32, device="cuda")
    return dict(table=table, lens=lens, refs=refs, moves=moves, count=count, pool=s["pool"])


def _plain_accept(s):
    page, n_pages, pool = s["case"]["page"], s["refs"].numel(), s["pool"]
    base = (s["lens"] - s["n_draft"]).long()
    nth = torch.arange(s["path"].shape[1], device=base.device)
    keep = nth < s["n_accept"][:, None]
    seq, j = keep.nonzero(as_tuple=True)
    src, dst = base[seq] + s["path"][seq, j], base[seq] + j
    row = pool[:, s["table"][seq, src // page].long(), :, src % page].clone()
    pool[:, s["table"][seq, dst // page].long(), :, dst % page] = row
    lens = (base + s["n_accept"]).to(torch.int32)
    at = torch.arange(s["table"].shape[1], device=base.device)
    kept = at < ((lens + page - 1) // page)[:, None]
    drop = ~kept & (at < ((s["lens"] + page - 1) // page)[:, None])
    refs = s["refs"] - _count_pages(s["table"], drop, n_pages)
    return dict(table=torch.where(kept, s["table"], -1), lens=lens, refs=refs, pool=pool)


def _plain_summarize(s):
    page = s["case"]["page"]
    at = torch.arange(s["table"].shape[1], device="cuda")
    seq, nth = ((at + 1) * page > s["first"][:, None]).logical_and(at * page < s["lens"][:, None]).nonzero(as_tuple=True)
    pages = s["table"][seq, nth].long()
    seen = nth[:, None] * page + torch.arange(page, device="cuda") < s["lens"][seq][:, None]
    k = s["k"][pages].float()
    code, scale = _bounds(k, seen[:, None].expand(k.shape[:-1]))
    s["codes"][pages], s["scales"][pages] = code, scale
    return dict(bounds=s["codes"] * s["scales"][..., None, None], scales=s["scales"])


def _softmax_sum(score, v):
    """Softmax of the last dimension times v, and the log of the sum; rows with nothing give zeros and -inf."""
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    return out, (torch.log(total) + torch.where(top == -math.inf, 0.0, top))[..., 0]


def _plain_tree(s):
    c, q = s["case"], s["q"]
    B, T, hq, D = q.shape
    G = hq // c["heads"]
    pages = s["table"].clamp(min=0).long()
    n = pages.shape[1] * c["page"]
    k = s["k"][pages].float().transpose(1, 2).reshape(B, c["heads"], n, D)
    v = s["v"][pages].float().transpose(1, 2).reshape(B, c["heads"], n, D)
    at = torch.arange(n, device="cuda")
    node = at - (s["lens"] - T)[:, None]
    word = s["mask"].gather(2, (node.clamp(0, T - 1) // 32)[:, None].expand(B, T, n))
    sees = (node < 0)[:, None] | (((word >> (node.clamp(0, T - 1) % 32)[:, None]) & 1 > 0) & (node < T)[:, None])
    rows = q.float().reshape(B, T, c["heads"], G, D).transpose(1, 2).reshape(B, c["heads"], T * G, D)
    score = torch.matmul(rows, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    score = torch.where(sees.repeat_interleave(G, 1)[:, None], score, -math.inf)
    v = torch.where((at < s["lens"][:, None])[:, None, :, None], v, 0.0)
    out, lse = _softmax_sum(score, v)
    out = out.reshape(B, c["heads"], T, G, D).transpose(1, 2).reshape(B, T, hq, D)
    return dict(out=out.to(q.dtype), lse=lse.reshape(B, c["heads"], T, G).transpose(1, 2).reshape(B, T, hq))


def _plain_sparse(s):
    c, q = s["case"], s["q"]
    B, T, hq, D = q.shape
    H, page, budget = c["heads"], c["page"], c["budget"]
    G = hq // H
    rows = q.float().reshape(B, T, H, G, D)
    amax = rows.abs().amax(-1).amax(-1)[..., None, None]
    fine = torch.isfinite(amax) & (amax >= 2.0**-100)
    code = torch.round(torch.where(fine, rows, 0.0) * torch.where(fine, 127.0 / torch.where(fine, amax, 1.0), 0.0))
    code = code.clamp(-127, 127)
    table = s["table"].clamp(min=0).long()
    n = table.shape[1]
    bound = s["codes"][table].float()  # [B, n, H, 2, D]
    both = torch.cat([code.clamp(max=0), code.clamp(min=0)], -1).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, 2 * D)
    part = torch.matmul(both, bound.permute(0, 2, 3, 4, 1).reshape(B, H, 2 * D, n))  # whole numbers below 2^24
    total = part.reshape(B, H, T, G, n).to(torch.int32).sum(3, dtype=torch.int32)
    scale = s["scales"][table].transpose(1, 2)[:, :, None]
    score = torch.where(torch.isinf(scale), math.inf, total.float() * scale).transpose(1, 2)  # [B, T, H, n]
    place = s["lens"][:, None] - T + torch.arange(T, device="cuda")  # the query's own position
    own_page = torch.div(place, page, rounding_mode="floor")[:, :, None, None]
    at = torch.arange(n, device="cuda")
    forced = (at < c["first"]) | (at > own_page - c["last"])
    order = torch.where(forced, math.inf, score)
    hidden = at > own_page
    # forced pages first, then by score; equal scores by the lower page
    rank = torch.sort(torch.where(hidden, -math.inf, order), descending=True, stable=True).indices
    group = torch.where(hidden, 2, torch.where(forced, 0, 1)).expand(B, T, H, n).gather(-1, rank)
    rank = rank.gather(-1, torch.sort(group, stable=True).indices)
    take = min(budget, n)
    chosen = rank[..., :take]
    chosen = torch.where(chosen <= own_page, chosen, n).sort(-1).values
    pages = torch.nn.functional.pad(torch.where(chosen < n, chosen, -1), (0, budget - take), value=-1)
    held = table[:, None, None].expand(B, T, H, n).gather(-1, chosen.clamp(max=n - 1))
    head = torch.arange(H, device="cuda")[:, None]
    k = s["k"][held, head].float().reshape(B, T, H, take * page, D)
    v = s["v"][held, head].float().reshape(B, T, H, take * page, D)
    spot = (chosen[..., None] * page + torch.arange(page, device="cuda")).reshape(B, T, H, take * page)
    sees = (spot <= place[:, :, None, None]) & (chosen < n).repeat_interleave(page, -1)
    score = torch.matmul(rows, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    score = torch.where(sees[:, :, :, None], score, -math.inf)
    out, lse = _softmax_sum(score, torch.where(sees[..., None], v, 0.0))
    return dict(out=out.reshape(B, T, hq, D).to(q.dtype), lse=lse.reshape(B, T, hq), pages=pages.to(torch.int32))


_plain = dict(fork=_plain_fork, retire=_plain_retire, accept=_plain_accept, summarize=_plain_summarize,
              tree=_plain_tree, sparse=_plain_sparse)


# --------------------------------------------------------------------------
# The same in 64 bits


def exact(case, seed):
    c = case
    if c["kind"] in ("fork", "retire", "accept"):
        return None  # whole numbers and copied bits: no rounding to compare
    s = prepare(case, seed)
    page, H = c["page"], c["heads"]
    table, lens = s["table"].tolist(), s["lens"].tolist()
    if c["kind"] == "summarize":
        scales = torch.zeros(s["scales"].shape, dtype=torch.float64, device="cuda")
        bounds = torch.zeros(s["codes"].shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            for j in range(max(0, n - c["fresh"]) // page, -(-n // page)):
                keys = s["k"][table[b][j], :, : min(page, n - j * page)].double()
                top = keys.abs().amax((1, 2))
                low, high = keys.amin(1), keys.amax(1)
                step = torch.where(top > 0, top / 127, 1.0)[:, None, None]
                bounds[table[b][j]] = torch.round(torch.stack([low, high], 1) / step) * step
                scales[table[b][j]] = top / 127
        return dict(bounds=bounds, scales=scales)
    B, T, hq, D = s["q"].shape
    G = hq // H
    out = torch.zeros(B, T, hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, hq), -math.inf, dtype=torch.float64, device="cuda")
    if c["kind"] == "tree":
        if 4.0 * sum(lens) * T * hq * D > 4e12:
            return None
        for b, n in enumerate(lens):
            held = torch.tensor(table[b][: -(-n // page)], device="cuda")
            spot = torch.arange(n, device="cuda")
            words = s["mask"][b].long() & 0xFFFFFFFF
            node = torch.arange(T, device="cuda")
            bits = (words[:, node // 32] >> (node % 32)) & 1
            sees = torch.cat([torch.ones(T, n - T, device="cuda", dtype=torch.bool), bits.bool()], 1)
            for h in range(H):
                keys = s["k"][held, h].double().reshape(-1, D)[spot]
                vals = s["v"][held, h].double().reshape(-1, D)[spot]
                for g in range(G):
                    w = s["q"][b, :, h * G + g].double() @ keys.T / math.sqrt(D)
                    w = w.masked_fill(~sees, -math.inf)
                    out[b, :, h * G + g] = torch.softmax(w, -1) @ vals
                    lse[b, :, h * G + g] = torch.logsumexp(w, -1)
        return dict(out=out, lse=lse)
    if B * T * H > 6000:
        return None
    # the choice of pages is whole-number arithmetic: codes of 32-bit products, whole sums, one 32-bit product
    codes = s["codes"].long()
    for b, n in enumerate(lens):
        width = -(-n // page)
        held = torch.tensor(table[b][:width], device="cuda")
        for h in range(H):
            lo, hi = codes[held, h, 0].double(), codes[held, h, 1].double()
            for t in range(T):
                place = n - T + t
                rows = s["q"][b, t, h * G : (h + 1) * G]
                top = rows.float().abs().max()
                qc = torch.round(rows.float() * (127.0 / top)).double().clamp(-127, 127)
                near = place // page
                total = (qc.clamp(min=0) @ hi[: near + 1].T + qc.clamp(max=0) @ lo[: near + 1].T).sum(0)
                score = total.float() * s["scales"][held[: near + 1], h]
                must = torch.arange(near + 1, device="cuda")
                must = (must < c["first"]) | (must > near - c["last"])
                left = c["budget"] - must.sum()
                best = torch.sort(score.masked_fill(must, -math.inf), descending=True, stable=True).indices
                place_in = torch.empty_like(best)
                place_in[best] = torch.arange(near + 1, device="cuda")
                chosen = (must | (place_in < left)).nonzero()[:, 0]
                spot = (chosen[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)
                seen = spot <= place
                keys = s["k"][held[chosen], h].double().reshape(-1, D)[seen]
                vals = s["v"][held[chosen], h].double().reshape(-1, D)[seen]
                w = rows.double() @ keys.T / math.sqrt(D)
                out[b, t, h * G : (h + 1) * G] = torch.softmax(w, -1) @ vals
                lse[b, t, h * G : (h + 1) * G] = torch.logsumexp(w, -1)
    return dict(out=out, lse=lse, pages=None)


# --------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c = case
    lens, page, H, D = _lens(c), c["page"], c["heads"], c["dim"]
    held = sum(-(-n // page) for n in lens)
    row = 2 * H * D
    width = max(-(-n // page) for n in lens)
    if c["kind"] in ("fork", "retire", "accept"):
        meta = 4 * (2 * c["seqs"] * (width + 1) + 2 * c["pages"])
        if c["kind"] == "fork":
            # a parent drawn c times gives c - 1 copies of its last page: about n/e sequences have no child
            moved = sum(n % page for n in lens) * math.exp(-1)
        elif c["kind"] == "retire":
            gone = max(1, c["seqs"] // 3) / c["seqs"]
            live = held * (1 - gone)
            moved = live * (1 - live / c["pages"]) * page
        else:
            depth = max(1, min(8, c["draft"] // 4))
            moved = c["seqs"] * (depth - 1) * depth / 2 / (depth + 1)
        return {"bytes": 2 * moved * row * c["pools"] + meta, "flops": 0}
    if c["kind"] == "summarize":
        new = sum(-(-n // page) - max(0, n - c["fresh"]) // page for n in lens)
        read = sum(n - max(0, n - c["fresh"]) // page * page for n in lens)
        return {"bytes": read * row + new * H * (2 * D + 4) + held * H * (2 * D + 4 + 8 * D), "flops": 3 * read * H * D}
    T, hq = c["draft"], c["qheads"]
    io = c["seqs"] * T * hq * (4 * D + 4) + 4 * held
    if c["kind"] == "tree":
        pairs = sum(T * (n - T) + T * (T + 1) / 2 for n in lens)
        return {"bytes": io + 2 * row * sum(lens) + 4 * c["seqs"] * T * (-(-T // 32)), "flops": 4 * pairs * hq * D}
    read, pairs, scored = 0, 0, 0
    for n in lens:
        seen = -(-n // page)
        per = min(c["budget"], seen)
        read += min(seen, per * T) * page
        pairs += T * min(per * page, n)
        scored += T * seen
    return {"bytes": io + 2 * row * read + held * H * (2 * D + 4) + 4 * c["seqs"] * T * H * c["budget"],
            "flops": 4 * pairs * hq * D + 2 * scored * hq * D}
