"""Cases of the operators for compact caches and drafted tokens: what is timed and compared.

Five kinds of pass, each as a serving program makes it:

store      new tokens' keys and values go into a paged cache held in 4 bits,
           and the values that they then stand for are read back
attend     attention of a tree of drafted tokens, of single tokens or of a
           prompt's chunk over a cache held in 4 bits
verify     drafted tokens are accepted or rejected by the target's and the
           draft's probabilities and given random numbers, and the next token is drawn
weigh      the attention weight that each cached token receives is added to
           what it has received so far
evict      the tokens of least accumulated weight are chosen to leave

`own = False` computes a pass by elementary torch operations in 32 bits,
`own = True` by the framework's entry points (host_transfer_gb300.kv).

A group of 32 elements of a token and head is held as 4-bit codes 1..15 and one
scale of the cache's type: s = (the group's largest magnitude) / 7 rounded to 5
significant bits, code = 8 + x / s rounded to whole and kept within 1..15; the
group stands for (code - 8) * s.
"""

import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
GROUP = 32  # elements that share a scale


# --------------------------------------------------------------------------
# Cases


def listed():
    return [
        # a decode step of a batch: one new token a sequence, latency counts
        dict(name="store_step", kind="store", seqs=32, fresh=1, heads=8, page=16, dim=128, dtype="bf16", layout="hnd",
             length=4096),
        # prompts that have just been computed, tokens-first pages, odd lengths
        dict(name="store_prompt", kind="store", seqs=4, fresh=8191, heads=8, page=64, dim=128, dtype="f16",
             layout="nhd", length=8191),
        # one sequence, one token, small pages: the latency of a decode step
        dict(name="attend_token", kind="attend", seqs=1, draft=1, qheads=32, heads=8, page=16, dim=128, dtype="bf16",
             layout="hnd", length=777),
        # a decode batch over long caches with grouped heads: the cache's bytes count
        dict(name="attend_batch", kind="attend", seqs=32, draft=1, qheads=64, heads=8, page=64, dim=128, dtype="bf16",
             layout="hnd", length=32768),
        # a verification step: trees of 13 drafted tokens, four query heads a key head
        dict(name="attend_tree", kind="attend", seqs=8, draft=13, qheads=32, heads=8, page=64, dim=128, dtype="bf16",
             layout="hnd", length=16384),
        # a chunk of a prompt over what came before; half precision, 64-wide heads, tokens-first pages
        dict(name="attend_chunk", kind="attend", seqs=2, draft=1023, qheads=32, heads=4, page=32, dim=64, dtype="f16",
             layout="nhd", length=16384),
        # one sequence's chain of four drafted tokens: latency counts
        dict(name="verify_chain", kind="verify", seqs=1, draft=4, vocab=32768, tree=False, certain=False),
        # trees of drafted tokens of a batch, large vocabulary
        dict(name="verify_trees", kind="verify", seqs=64, draft=15, vocab=131072, tree=True, certain=False),
        # a decode batch over a cache held in 4 bits
        dict(name="weigh_batch", kind="weigh", seqs=32, draft=1, qheads=32, heads=8, page=64, dim=128, dtype="bf16",
             layout="hnd", length=16384, four=True),
        # a chunk of a prompt over a cache held in 16 bits
        dict(name="weigh_chunk", kind="weigh", seqs=2, draft=511, qheads=32, heads=8, page=64, dim=128, dtype="bf16",
             layout="hnd", length=8192, four=False),
        # a decode step's end: a few tokens over the budget leave
        dict(name="evict_step", kind="evict", seqs=8, length=2063, budget=2048, first=4, last=256),
        # after long prompts: most tokens leave
        dict(name="evict_prompt", kind="evict", seqs=32, length=65521, budget=8192, first=4, last=1024),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["store", "attend", "attend", "attend", "verify", "verify", "weigh", "evict"])
    if kind == "verify":
        c = dict(kind=kind, seqs=_spread(rng, 1, 64), draft=_spread(rng, 1, 24), vocab=_spread(rng, 100, 131072),
                 tree=rng.choice([True, False]), certain=rng.choice([True, False, False]))
        while c["seqs"] > 1 and c["seqs"] * (c["draft"] + 1) * c["vocab"] > 64 * 16 * 131072:
            c["seqs"] //= 2
        return c
    if kind == "evict":
        c = dict(kind=kind, seqs=_spread(rng, 1, 32), length=_spread(rng, 2, 65536), first=rng.choice([0, 1, 4, 16]))
        c["last"] = _spread(rng, 1, 512)
        c["budget"] = c["first"] + c["last"] + _spread(rng, 1, 8192)
        return c
    c = dict(kind=kind, dtype=rng.choice(["bf16", "f16"]), layout=rng.choice(["hnd", "nhd"]),
             page=rng.choice([16, 16, 24, 32, 64, 128]), dim=rng.choice([64, 96, 128, 128, 256]),
             heads=rng.choice([1, 2, 4, 8, 32]), seqs=_spread(rng, 1, 32), length=_spread(rng, 1, 32768))
    if kind == "store":
        c["fresh"] = rng.choice([1, _spread(rng, 1, c["length"])])
        while c["seqs"] > 1 and c["seqs"] * c["heads"] * c["fresh"] * c["dim"] > 4 * 8 * 8191 * 128:
            c["seqs"] //= 2
        while c["heads"] > 1 and c["seqs"] * c["heads"] * c["fresh"] * c["dim"] > 4 * 8 * 8191 * 128:
            c["heads"] //= 2
    else:
        c["qheads"] = c["heads"] * rng.choice([g for g in (1, 2, 4, 7, 8, 16) if g * c["heads"] <= 64])
        c["draft"] = rng.choice([1, _spread(rng, 1, 64), _spread(rng, 64, 512) if kind == "attend" else 1])
        c["length"] = max(c["length"], c["draft"])
        if kind == "weigh":
            c["four"] = rng.choice([True, False])
        while c["seqs"] > 1 and c["seqs"] * c["draft"] * c["qheads"] * c["length"] > 2 * 1023 * 32 * 8192:
            c["seqs"] //= 2
        while c["length"] > 2 * c["draft"] and c["draft"] * c["qheads"] * c["length"] > 2 * 1023 * 32 * 8192:
            c["length"] //= 2
    while c["seqs"] > 1 and c["seqs"] * c["heads"] * c["length"] * c["dim"] > 32 * 8 * 16384 * 128:
        c["seqs"] //= 2
    return c


def _lens(c):
    """Lengths of a ragged batch: the first sequence is the longest, the others at least three tenths of it."""
    low = c.get("draft", c.get("fresh", 1))
    return [max(low, c["length"] - int(0.7 * c["length"] * ((i * 0.6180339887) % 1.0))) for i in range(c["seqs"])]


# --------------------------------------------------------------------------
# Inputs


def _pool(shape, layout, dtype):
    """Pages [pages, heads, tokens, ...] whose memory is in that order, or tokens before heads."""
    pages, heads, page, dim = shape
    if layout == "hnd":
        return torch.empty(shape, dtype=dtype, device="cuda")
    return torch.empty((pages, page, heads, dim), dtype=dtype, device="cuda").transpose(1, 2)


def _table(c, lens, n_pages, gen):
    """Page table and lengths; the pages are drawn without order from the pool."""
    need = [-(-n // c["page"]) for n in lens]
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    need_t = torch.tensor(need, device="cuda")
    at = torch.arange(max(need), device="cuda")
    base = torch.cumsum(need_t, 0) - need_t
    table = torch.where(at < need_t[:, None], order[(base[:, None] + at).clamp(max=n_pages - 1)], -1)
    return table.to(torch.int32).contiguous(), torch.tensor(lens, dtype=torch.int32, device="cuda")


def _quantise(x, dtype):
    """Codes (whole numbers 1..15, as x) and scales of x [..., dim], given in 32 bits."""
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    top = g.abs().amax(-1)
    bits = (top / torch.full_like(top, 7.0)).view(torch.int32)
    step = ((bits + 0x3FFFF + ((bits >> 19) & 1)) & -0x80000).view(torch.float32)  # 5 significant bits
    step = torch.where(step < 2.0**-100, 0.0, step).clamp(max=2.0**121).to(dtype).float()
    fine = torch.isfinite(g).all(-1)
    code = torch.round(g / torch.where(step > 0, step, 1.0)[..., None]).clamp(-7, 7)
    code = torch.where((fine & (step > 0))[..., None], code, 0.0) + 8
    return code.reshape(x.shape), torch.where(fine, step, math.nan).to(dtype)


def _pack(code):
    """Two codes a byte, the even element in the low half."""
    pair = code.to(torch.uint8).reshape(*code.shape[:-1], -1, 2)
    return pair[..., 0] | (pair[..., 1] << 4)


def _unpack(codes, scales):
    """The values that codes and scales stand for, in 32 bits."""
    code = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1).float() - 8
    return (code.reshape(*code.shape[:-1], -1, GROUP) * scales.float()[..., None]).reshape(code.shape)


def _fill(pages, gen, c, shared):
    """Normal values; those of one page and head share a direction where `shared` (keys)."""
    n, H, page, D = pages.shape
    wide = torch.empty(H, 1, 1, device="cuda").uniform_(0.5, 2.0, generator=gen)
    for at in range(0, n, 1024):
        x = torch.randn((min(1024, n - at), H, page, D), generator=gen, device="cuda")
        if shared:
            x = (x + torch.randn((x.shape[0], H, 1, D), generator=gen, device="cuda")) * wide
        yield slice(at, at + x.shape[0]), x.to(DT[c["dtype"]])


def _cache(c, n_pages, gen, shared):
    """A pool in 4 bits: (codes, scales)."""
    shape = (n_pages, c["heads"], c["page"])
    codes = _pool((*shape, c["dim"] // 2), c["layout"], torch.uint8)
    scales = _pool((*shape, c["dim"] // GROUP), c["layout"], DT[c["dtype"]])
    for part, x in _fill(torch.empty((*shape, c["dim"]), device="meta"), gen, c, shared):
        code, scales[part] = _quantise(x.float(), DT[c["dtype"]])
        codes[part] = _pack(code)
    return codes, scales


def _mask(seqs, T, gen):
    """Bits of a random tree: each node's parent is one of the last eight before it, or the context's last token."""
    at = torch.arange(T, device="cuda")
    back = torch.randint(1, 9, (seqs, T), generator=gen, device="cuda")
    reach = torch.eye(T, dtype=torch.bool, device="cuda").repeat(seqs, 1, 1)
    reach |= (at[None, :, None] - back[:, :, None]) == at[None, None, :]
    for _ in range(max(1, T.bit_length())):
        reach = torch.bmm(reach.float(), reach.float()) > 0
    bits = torch.nn.functional.pad(reach, (0, -T % 32)).reshape(seqs, T, -1, 32).long()
    words = (bits << torch.arange(32, device="cuda")).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 2654435761 % (1 << 62) + 1)
    if c["kind"] == "verify":
        return _prepare_verify(c, gen)
    if c["kind"] == "evict":
        # attention weight is spread over many decades; tokens that nobody has looked at have none
        lens = torch.tensor(_lens(c), dtype=torch.int32, device="cuda")
        weight = torch.exp(2.5 * torch.randn(c["seqs"], c["length"], generator=gen, device="cuda"))
        weight *= torch.rand(weight.shape, generator=gen, device="cuda") > 0.03
        return dict(case=c, lens=lens, weight=weight)
    dt, lens = DT[c["dtype"]], _lens(c)
    n_pages = sum(-(-n // c["page"]) for n in lens) + 5
    table, lens_t = _table(c, lens, n_pages, gen)
    s = dict(case=c, table=table, lens=lens_t)
    if c["kind"] == "store":
        shape = (c["seqs"], c["fresh"], c["heads"], c["dim"])
        s["k"] = (torch.randn(shape, generator=gen, device="cuda") * 1.5).to(dt)
        s["v"] = torch.randn(shape, generator=gen, device="cuda").to(dt)
        for name in ("k4", "v4"):
            codes = _pool((n_pages, c["heads"], c["page"], c["dim"] // 2), c["layout"], torch.uint8).fill_(0x88)
            s[name] = codes, _pool((n_pages, c["heads"], c["page"], c["dim"] // GROUP), c["layout"], dt).zero_()
        return s
    T = c["draft"]
    s["q"] = torch.randn(c["seqs"], T, c["qheads"], c["dim"], generator=gen, device="cuda").to(dt)
    # prompts and single tokens see what comes before them, drafts are trees
    s["mask"] = _mask(c["seqs"], T, gen) if 1 < T <= 64 else None
    if c["kind"] == "attend" or c["four"]:
        s["k"] = _cache(c, n_pages, gen, True)
    else:
        s["k"] = _pool((n_pages, c["heads"], c["page"], c["dim"]), c["layout"], dt)
        for part, x in _fill(s["k"], gen, c, True):
            s["k"][part] = x
    if c["kind"] == "attend":
        s["v"] = _cache(c, n_pages, gen, False)
    else:
        s["lse"] = torch.empty(c["seqs"], T, c["qheads"], device="cuda")
        for b in range(c["seqs"]):  # what the attention of the same step has returned
            score, sees = _scores(s, slice(b, b + 1), lens[b])
            s["lse"][b] = _rows_back(torch.logsumexp(score.masked_fill(~sees, -math.inf), -1)[..., None], c)[0, ..., 0]
        s["weight"] = torch.rand(c["seqs"], table.shape[1] * c["page"], generator=gen, device="cuda")
    return s


def _prepare_verify(c, gen):
    B, T, V = c["seqs"], c["draft"], c["vocab"]
    logits = torch.randn(B, T + 1, V, generator=gen, device="cuda") * 3
    q = torch.softmax(logits[:, :T], -1)
    p = torch.softmax(logits + torch.randn(B, T + 1, V, generator=gen, device="cuda") * 0.7, -1)
    at = torch.arange(T, device="cuda", dtype=torch.int32)
    parents = at.expand(B, T) - 1
    if c["tree"]:
        back = torch.randint(1, 4, (B, T), generator=gen, device="cuda", dtype=torch.int32)
        parents = (at - back).clamp(min=-1)
    rows = torch.gather(q, 1, (parents.long() + 1)[..., None].expand(B, T, V))
    if c["certain"]:  # the draft proposes its best tokens, and no two alike for one parent
        rank = (torch.tril(parents[:, :, None] == parents[:, None, :], -1)).sum(-1)
        best = torch.topk(rows, min(8, V), -1).indices
        tokens = best.gather(-1, rank.clamp(max=best.shape[-1] - 1)[..., None])[..., 0]
    else:
        noise = torch.empty_like(rows).exponential_(generator=gen)
        tokens = (rows / noise.clamp(min=1e-30)).argmax(-1)
    u = torch.rand(B, T + 1, generator=gen, device="cuda")
    return dict(case=c, p=p, q=None if c["certain"] else q, tokens=tokens.to(torch.int32).contiguous(), u=u,
                parents=parents.contiguous() if c["tree"] else None)


# --------------------------------------------------------------------------
# One pass


def run(state):
    return (_own if own else _plain)[state["case"]["kind"]](state)


def _own_store(s):
    from host_transfer_gb300 import kv

    kv.ibp_kv4_store(s["k"], s["v"], s["k4"], s["v4"], s["table"], s["lens"])
    k, v = kv.ibp_kv4_load(s["k4"], s["v4"], s["table"], s["lens"], s["case"]["fresh"])
    return dict(k=k, v=v, k_scales=s["k4"][1], v_scales=s["v4"][1])


def _own_attend(s):
    from host_transfer_gb300 import kv

    out, lse = kv.ibp_kv4_attention(s["q"], s["k"], s["v"], s["table"], s["lens"], mask=s["mask"])
    return dict(out=out, lse=lse)


def _own_verify(s):
    from host_transfer_gb300 import kv

    path, n_accept, token = kv.ibp_kv_verify(s["p"], s["tokens"], s["u"], q=s["q"], parents=s["parents"])
    return dict(path=path, n_accept=n_accept, token=token)


def _own_weigh(s):
    from host_transfer_gb300 import kv

    return dict(weight=kv.ibp_kv_weigh(s["q"], s["k"], s["table"], s["lens"], s["lse"], s["weight"], mask=s["mask"],
                                       decay=0.96875))


def _own_evict(s):
    from host_transfer_gb300 import kv

    c = s["case"]
    path, n_draft, n_keep, weight = kv.ibp_kv_evict(s["weight"], s["lens"], c["budget"], keep_first=c["first"],
                                                    keep_last=c["last"])
    return dict(path=path, n_draft=n_draft, n_keep=n_keep, weight=weight)


_own = dict(store=_own_store, attend=_own_attend, verify=_own_verify, weigh=_own_weigh, evict=_own_evict)


def _plain_store(s):
    c = s["case"]
    spot = (s["lens"] - c["fresh"])[:, None] + torch.arange(c["fresh"], device="cuda")
    page = s["table"].gather(1, spot // c["page"]).long()
    slot = spot % c["page"]
    back = []
    for x, (codes, scales) in ((s["k"], s["k4"]), (s["v"], s["v4"])):
        code, scale = _quantise(x.float(), x.dtype)
        codes[page, :, slot] = _pack(code)
        scales[page, :, slot] = scale
        back.append(_unpack(codes[page, :, slot], scales[page, :, slot]).to(x.dtype))
    return dict(k=back[0], v=back[1], k_scales=s["k4"][1], v_scales=s["v4"][1])


def _values(pages, held):
    """[seqs, pages, heads, tokens, dim] of the held pages, in 32 bits."""
    return _unpack(pages[0][held], pages[1][held]) if isinstance(pages, tuple) else pages[held].float()


def _scores(s, rows, width):
    """Scores [seqs, heads, T * group, width] of the given sequences, and which of them a query sees."""
    c = s["case"]
    q, lens = s["q"][rows], s["lens"][rows]
    B, T, hq, D = q.shape
    H, G = c["heads"], hq // c["heads"]
    held = s["table"][rows, : -(-width // c["page"])].clamp(min=0).long()
    n = held.shape[1] * c["page"]
    k = _values(s["k"], held).transpose(1, 2).reshape(B, H, n, D)
    q = q.float().reshape(B, T, H, G, D).transpose(1, 2).reshape(B, H, T * G, D)
    score = torch.matmul(q, k.transpose(-1, -2)) * (1 / math.sqrt(D))
    at = torch.arange(n, device="cuda")
    node = (at - (lens - T)[:, None])[:, None]
    if s["mask"] is None:
        sees = node <= torch.arange(T, device="cuda")[:, None]
    else:
        word = s["mask"][rows].gather(2, (node.clamp(0, T - 1) // 32).expand(B, T, n))
        sees = (node < 0) | (((word >> (node.clamp(0, T - 1) % 32)) & 1 > 0) & (node < T))
    return score, sees.repeat_interleave(G, 1)[:, None]


def _rows_back(x, c):
    """[seqs, heads, T * group, ...] to [seqs, T, q_heads, ...]."""
    B, H, rows, D = x.shape
    T = c["draft"]
    return x.reshape(B, H, T, rows // T, D).transpose(1, 2).reshape(B, T, -1, D)


def _plain_attend(s):
    c = s["case"]
    score, sees = _scores(s, slice(None), c["length"])
    held = s["table"].clamp(min=0).long()
    v = _values(s["v"], held).transpose(1, 2)
    v = v.reshape(v.shape[0], v.shape[1], -1, v.shape[-1])
    v = torch.where((torch.arange(v.shape[2], device="cuda") < s["lens"][:, None])[:, None, :, None], v, 0.0)
    score = torch.where(sees, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / total
    return dict(out=_rows_back(out, c).to(s["q"].dtype), lse=_rows_back(torch.log(total) + top, c)[..., 0])


def _plain_verify(s):
    p = torch.nan_to_num(s["p"], nan=0.0).clamp(0, 1)
    q = None if s["q"] is None else torch.nan_to_num(s["q"], nan=0.0).clamp(0, 1)
    B, T = s["tokens"].shape
    V = p.shape[-1]
    every = torch.arange(B, device="cuda")
    node = torch.full((B,), -1, dtype=torch.int32, device="cuda")
    path = torch.full((B, T), -1, dtype=torch.int32, device="cuda")
    count = torch.zeros(B, dtype=torch.int32, device="cuda")
    left = draw_from = p[:, 0]
    ids = torch.arange(V, device="cuda")
    for t in range(T):
        x = s["tokens"][:, t].long()
        tried = (s["parents"][:, t] if s["parents"] is not None else torch.full_like(node, t - 1)) == node
        # what the token was drawn from: its parent's row, or certainty
        drawn = (ids == x[:, None]).float() if q is None else q[every, (node.long() + 1).clamp(max=T - 1)]
        ok = tried & (s["u"][:, t].double() * drawn[every, x].double() < left[every, x].double())
        rest = (left - drawn).clamp(min=0)
        total = torch.round(rest * 2.0**44).long().sum(1)
        lost = (tried & ~ok & (total > 0))[:, None]
        scaled = rest * (2.0**44 / total.double()).float()[:, None]
        left = torch.where(ok[:, None], p[:, t + 1], torch.where(lost, scaled, left))
        draw_from = torch.where(ok[:, None], p[:, t + 1], torch.where(lost, rest, draw_from))
        path = torch.where(ok[:, None] & (torch.arange(T, device="cuda") == count[:, None]), t, path)
        count = count + ok.to(torch.int32)
        node = torch.where(ok, t, node).to(torch.int32)
    weight = torch.round(draw_from * 2.0**44).long()
    total = weight.sum(1)
    aim = torch.minimum((s["u"][:, T].double() * total.double()).floor().long(), total - 1)
    token = (torch.cumsum(weight, 1) <= aim[:, None]).sum(1)
    return dict(path=path.to(torch.int32), n_accept=count, token=torch.where(total > 0, token, -1).to(torch.int32))


def _plain_weigh(s):
    c = s["case"]
    T, n = c["draft"], s["weight"].shape[1]
    score, sees = _scores(s, slice(None), n)
    lse = s["lse"].reshape(c["seqs"], T, c["heads"], -1).transpose(1, 2).reshape(c["seqs"], c["heads"], -1, 1)
    got = torch.where(sees, torch.exp(score - lse), 0.0).sum((1, 2))
    at = torch.arange(n, device="cuda")
    before = torch.where(at < (s["lens"] - T)[:, None], s["weight"] * 0.96875, 0.0)
    return dict(weight=torch.where(at < s["lens"][:, None], before + got, s["weight"]))


def _plain_evict(s):
    c, weight = s["case"], s["weight"]
    B, n = weight.shape
    at = torch.arange(n, device="cuda")
    lens = s["lens"][:, None]
    # by weight, the earlier first when equal; then the ones that stay in any case before the others
    rank = torch.sort(weight, descending=True, stable=True).indices
    group = torch.where(at >= lens, 2, torch.where((at < c["first"]) | (at >= lens - c["last"]), 0, 1))
    rank = rank.gather(1, torch.sort(group.gather(1, rank), stable=True).indices)
    take = min(c["budget"], n)
    kept = rank[:, :take].sort(1).values
    over = lens > c["budget"]
    path = torch.nn.functional.pad(torch.where(over, kept, -1), (0, c["budget"] - take), value=-1).to(torch.int32)
    moved = torch.nn.functional.pad(weight.gather(1, kept), (0, n - take))
    out = torch.where(over, moved, torch.where(at < lens, weight, 0.0))
    return dict(path=path, n_draft=torch.where(over, lens, 0)[:, 0].to(torch.int32),
                n_keep=torch.where(over, c["budget"], 0)[:, 0].to(torch.int32), weight=out)


_plain = dict(store=_plain_store, attend=_plain_attend, verify=_plain_verify, weigh=_plain_weigh, evict=_plain_evict)


# --------------------------------------------------------------------------
# The same in 64 bits


def _decoded(pages, held, head, D):
    """Rows [tokens, dim] of a head's held pages, in 64 bits."""
    if not isinstance(pages, tuple):
        return pages[held, head].double().reshape(-1, D)
    codes = pages[0][held, head].reshape(-1, D // 2).long()
    code = torch.empty(codes.shape[0], D, dtype=torch.float64, device="cuda")
    code[:, 0::2], code[:, 1::2] = (codes % 16 - 8).double(), (codes // 16 - 8).double()
    return code * pages[1][held, head].reshape(-1, D // GROUP).double().repeat_interleave(GROUP, 1)


def exact(case, seed):
    c = case
    if c["kind"] == "verify":
        return None  # whole numbers: no rounding to compare
    s = prepare(case, seed)
    if c["kind"] == "evict":
        weight = torch.zeros(s["weight"].shape, dtype=torch.float64)
        for b, n in enumerate(s["lens"].tolist()):
            w = s["weight"][b, :n].cpu().tolist()
            inner = range(min(c["first"], n), max(min(c["first"], n), n - c["last"]))
            spare = c["budget"] - (n - len(inner))  # places for tokens that do not stay in any case
            gone = sorted(inner, key=lambda i: (-w[i], i))[spare:] if n > c["budget"] else []
            kept = torch.ones(n, dtype=torch.bool)
            kept[gone] = False
            weight[b, : int(kept.sum())] = torch.tensor(w, dtype=torch.float64)[kept]
        return dict(path=None, n_draft=None, n_keep=None, weight=weight.cuda())
    page, H, D = c["page"], c["heads"], c["dim"]
    if c["kind"] == "store":
        out = dict(k=None, v=None, k_scales=None, v_scales=None)
        for name in ("k", "v"):
            x = s[name].double().unflatten(-1, (-1, GROUP))
            top = x.abs().amax(-1, keepdim=True)
            top = top / torch.full_like(top, 7.0)
            part, power = torch.frexp(top)  # part in [1/2, 1): its first 5 bits
            step = torch.round(part * 32) / 32
            for bit in range(8):  # times 2^power, exactly
                by = 2.0 ** (1 << bit)
                step = torch.where((power.abs() >> bit) & 1 > 0, torch.where(power < 0, step * (1 / by), step * by), step)
            step = step if c["dtype"] == "bf16" else torch.round(step * 2.0**24) / 2.0**24
            code = torch.round(x / torch.where(step > 0, step, 1.0)).clamp(-7, 7)
            out[name] = (code * step).flatten(-2)
        return out
    T, hq = c["draft"], c["qheads"]
    G = hq // H
    lens, table = s["lens"].tolist(), s["table"].tolist()
    if 4.0 * sum(lens) * T * hq * D > 4e12:
        return None
    attend = c["kind"] == "attend"
    out = torch.zeros(c["seqs"], T, hq, D if attend else 1, dtype=torch.float64, device="cuda")
    lse = torch.full((c["seqs"], T, hq), -math.inf, dtype=torch.float64, device="cuda")
    weight = None if attend else s["weight"].double()
    node = torch.arange(T, device="cuda")
    for b, n in enumerate(lens):
        held = torch.tensor(table[b][: -(-n // page)], device="cuda")
        if s["mask"] is None:
            bits = node[:, None] >= node
        else:
            bits = (((s["mask"][b].long() & 0xFFFFFFFF)[:, node // 32] >> (node % 32)) & 1).bool()
        sees = torch.cat([torch.ones(T, n - T, device="cuda", dtype=torch.bool), bits], 1)
        if not attend:
            weight[b, : n - T] *= 0.96875
            weight[b, n - T : n] = 0
        for h in range(H):
            keys = _decoded(s["k"], held, h, D)[:n]
            vals = _decoded(s["v"], held, h, D)[:n] if attend else None
            for g in range(h * G, h * G + G):
                w = (s["q"][b, :, g].double() @ keys.T / math.sqrt(D)).masked_fill(~sees, -math.inf)
                if attend:
                    out[b, :, g] = torch.softmax(w, -1) @ vals
                    lse[b, :, g] = torch.logsumexp(w, -1)
                else:
                    weight[b, :n] += torch.exp(w - s["lse"][b, :, g, None].double()).sum(0)
    return dict(out=out, lse=lse) if attend else dict(weight=weight)


# --------------------------------------------------------------------------
# What a pass cannot do without


def work(case):
    c = case
    if c["kind"] == "verify":
        # single probabilities of the tokens tried, and the rows of the last one: one of the target's, one of the draft's
        rows = c["seqs"] * c["vocab"] * 4
        return {"bytes": rows * (1 if c["certain"] else 2) + c["seqs"] * c["draft"] * 24, "flops": 4 * rows / 4}
    lens = _lens(c)
    if c["kind"] == "evict":
        return {"bytes": 4 * sum(lens) + c["seqs"] * (4 * c["length"] + 4 * c["budget"]), "flops": 0}
    H, D, page = c["heads"], c["dim"], c["page"]
    four = D // 2 + 2 * (D // GROUP)  # bytes of a token and head in 4 bits, its scales among them
    held = sum(-(-n // page) for n in lens)
    if c["kind"] == "store":
        new = c["seqs"] * c["fresh"] * H
        return {"bytes": 2 * new * (2 * D + four + 2 * D), "flops": 8 * new * D}
    T, hq = c["draft"], c["qheads"]
    pairs = sum(T * (n - T) + T * (T + 1) / 2 for n in lens)
    mask = 4 * c["seqs"] * T * (-(-T // 32)) if 1 < T <= 64 else 0
    if c["kind"] == "attend":
        return {"bytes": 2 * four * H * sum(lens) + c["seqs"] * T * hq * (4 * D + 4) + 4 * held + mask,
                "flops": 4 * pairs * hq * D}
    row = four if c["four"] else 2 * D
    return {"bytes": row * H * sum(lens) + c["seqs"] * T * hq * (2 * D + 4) + 4 * held + mask + 8 * sum(lens),
            "flops": 2 * pairs * hq * D}
