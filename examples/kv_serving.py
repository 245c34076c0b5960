"""A decode step of one layer on a compressed, paged key/value cache.

The prompt's keys and values lie compressed in pinned host memory, as
``bench.py --config llm`` holds them.  The step

1. decodes them with the rows in page order (ibp_gather_decompress) and copies
   the result into the pages of an HBM pool,
2. summarises the pages' keys and lets each sequence's last token attend to the
   few pages that score highest (ibp_kv_summarize, ibp_sparse_attention),
3. forks each sequence into beams (ibp_kv_fork, ibp_kv_copy), appends a tree of
   drafted tokens to every beam and attends to it (ibp_tree_attention),
4. keeps an accepted path of each beam (ibp_kv_accept), frees the losing beams
   (ibp_kv_free) and compacts the pool (ibp_kv_compact, ibp_kv_copy).

    python examples/kv_serving.py [--seq 1024] [--heads 8] [--beams 3]
"""

from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import numpy as np  # noqa: E402
import torch  # noqa: E402

from host_transfer_gb300 import ibp, kv, workloads  # noqa: E402

DIM = 128


def compressed_cache(seq: int, heads: int, layer: int):
    """One layer's K and V in pinned host memory, each compressed in place with
    a plan of its own."""
    tables = []
    for words in workloads.llm_kv(layer, heads=heads, seq=seq, head_dim=DIM):
        rows = torch.empty(words.shape, dtype=torch.int32, pin_memory=True)
        rows.numpy()[...] = words.view(np.int32)
        plan = ibp.ibp_plan_create(*ibp.ibp_preprocess(rows[: min(len(rows), 4096)].cuda(), 0.99))
        _, bitmask, _ = ibp.ibp_compress(plan, rows)
        tables.append((plan, rows, bitmask))
    return tables


def decode_into(pool: torch.Tensor, table, pages: torch.Tensor, seq: int):
    """Decodes a compressed cache and copies it into the given pages of a pool [n_pages,
    heads, page_tokens, dim]: row (head, position) of the table becomes its page's row."""
    plan, slots, bitmask = table
    _, heads, page, _ = pool.shape
    at = torch.arange(len(pages) * page, device="cuda").clamp(max=seq - 1).reshape(len(pages), 1, page)
    rows = torch.arange(heads, device="cuda").reshape(1, heads, 1) * seq + at
    out = ibp.ibp_gather_decompress(plan, slots, bitmask, rows.reshape(-1).contiguous())
    ibp.ibp_get_status(plan)
    pool[pages.long()] = out.view(pool.dtype).reshape(len(pages), heads, page, DIM)


def append(pool: torch.Tensor, table, lens, refs, rows):
    """Appends rows [2, n_seqs, T, heads, dim] to every sequence: takes the lowest
    free pages for those that grow past their last one.  Plain torch, which reads
    their number back to the host."""
    n_seqs, T, page = rows.shape[1], rows.shape[2], pool.shape[3]
    before, after = (lens + page - 1) // page, (lens + T + page - 1) // page
    place = torch.arange(table.shape[1], device="cuda")
    grows = (place >= before[:, None]) & (place < after[:, None])
    fresh = (refs == 0).nonzero()[: int(grows.sum()), 0].to(torch.int32)
    table[grows] = fresh
    refs[fresh.long()] = 1
    at = lens[:, None].long() + torch.arange(T, device="cuda")
    pages = table.gather(1, at // page).long()
    pool[:, pages, :, at % page] = rows.permute(1, 2, 0, 3, 4).to(pool.dtype)
    lens += T


def tree_mask(parents: list[int], n_seqs: int) -> torch.Tensor:
    """Words of ibp_tree_attention for one tree, the same for every sequence."""
    bits = []
    for t, parent in enumerate(parents):
        bits.append((bits[parent] if parent >= 0 else 0) | 1 << t)
    words = [[(b >> 32 * w) & 0xFFFFFFFF for w in range((len(parents) + 31) // 32)] for b in bits]
    return torch.from_numpy(np.array(words, np.uint32).view(np.int32)).cuda().expand(n_seqs, -1, -1).contiguous()


def run(seq: int = 1024, heads: int = 8, group: int = 4, page: int = 64, beams: int = 3, budget: int = 6, seed: int = 0):
    """Returns what the checks of the step need: inputs and outputs by name."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    n_seqs, prompt_pages = 2, -(-seq // page)
    n_pages = n_seqs * prompt_pages + 2 * n_seqs * beams + 8
    # K and V of the layer are two pools that share their page ids
    pool = torch.zeros((2, n_pages, heads, page, DIM), dtype=torch.bfloat16, device="cuda")
    k, v = pool[0], pool[1]
    lens = torch.tensor([seq, seq - page // 2], dtype=torch.int32, device="cuda")
    table = torch.full((n_seqs, prompt_pages + 2), -1, dtype=torch.int32, device="cuda")
    table[:, :prompt_pages] = torch.randperm(n_pages, generator=gen, device="cuda")[: n_seqs * prompt_pages].reshape(
        n_seqs, -1).to(torch.int32)
    held = torch.arange(table.shape[1], device="cuda") < ((lens + page - 1) // page)[:, None]
    table.masked_fill_(~held, -1)
    refs = torch.zeros(n_pages, dtype=torch.int32, device="cuda")
    refs[table[held].long()] = 1

    for b in range(n_seqs):
        pages = table[b][held[b]]
        for p, t in zip(pool, compressed_cache(seq, heads, layer=b)):
            decode_into(p, t, pages, seq)

    codes = torch.zeros((n_pages, heads, 2, DIM), dtype=torch.int8, device="cuda")
    scales = torch.zeros((n_pages, heads), device="cuda")
    kv.ibp_kv_summarize(k, table, lens, codes, scales)
    q1 = torch.randn((n_seqs, 1, heads * group, DIM), generator=gen, device="cuda").bfloat16()
    sparse = kv.ibp_sparse_attention(q1, k, v, table, lens, codes, scales, budget, keep_first=1, keep_last=2)
    first = dict(q=q1, k=k.clone(), v=v.clone(), table=table, lens=lens.clone(), codes=codes.clone(),
                 scales=scales.clone(), out=sparse[0], lse=sparse[1], pages=sparse[2], budget=budget)

    parents = torch.arange(n_seqs, device="cuda", dtype=torch.int32).repeat_interleave(beams)
    table, lens, refs, moves, count = kv.ibp_kv_fork(table, lens, refs, parents, page)
    kv.ibp_kv_copy(pool, moves, count)

    tree = [-1, -1, -1, 0, 0, 1, 3, 3, 4, 6]  # three first candidates, deeper nodes behind them
    T, n = len(tree), len(parents)
    append(pool, table, lens, refs, torch.randn((2, n, T, heads, DIM), generator=gen, device="cuda"))
    q = torch.randn((n, T, heads * group, DIM), generator=gen, device="cuda").bfloat16()
    mask = tree_mask(tree, n)
    out, lse = kv.ibp_tree_attention(q, k, v, table, lens, mask=mask)
    second = dict(q=q, k=k.clone(), v=v.clone(), table=table.clone(), lens=lens.clone(), mask=mask, out=out, lse=lse)

    n_draft = torch.full((n,), T, dtype=torch.int32, device="cuda")
    path = torch.tensor([[0, 3, 6, 9]], dtype=torch.int32, device="cuda").repeat(n, 1)
    n_accept = (torch.arange(n, device="cuda", dtype=torch.int32) % 4) + 1
    table, lens, refs = kv.ibp_kv_accept(pool, table, lens, refs, n_draft, path, n_accept, inplace=True)

    losers = torch.tensor([i for i in range(n) if i % beams], dtype=torch.int32, device="cuda")
    table, lens, refs = kv.ibp_kv_free(table, lens, refs, losers, page, inplace=True)
    before = dict(pool=pool.clone(), table=table.clone())
    table, refs, moves, count = kv.ibp_kv_compact(table, refs, page, inplace=True)
    kv.ibp_kv_copy(pool, moves, count)
    kv.ibp_kv_get_status()
    return dict(first=first, second=second, before=before, pool=pool, table=table, lens=lens, refs=refs,
                moved=int(count.item()), page=page)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--seq", type=int, default=1024)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--beams", type=int, default=3)
    a = ap.parse_args()
    r = run(seq=a.seq, heads=a.heads, beams=a.beams)
    live = int((r["refs"] > 0).sum())
    print(f"pages attended per query: {r['first']['pages'].shape[-1]} of {-(-a.seq // r['page'])}")
    print(f"lengths after acceptance: {r['lens'].tolist()}")
    print(f"live pages: {live}, moved by compaction: {r['moved']}, highest live page: {int(r['refs'].nonzero().max())}")


if __name__ == "__main__":
    main()
