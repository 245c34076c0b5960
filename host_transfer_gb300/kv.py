"""Python binding of libibp's paged key/value cache operators (ctypes).

Argument marshalling only, as in ``host_transfer_gb300.ibp``: every step runs
in the library's CUDA kernels.  Names and formulas follow include/ibp.h:

    table, lens, refs, moves, count = ibp_kv_fork(table, lens, refs, parents, page_tokens)
    table, lens, refs = ibp_kv_free(table, lens, refs, seqs, page_tokens)
    table, refs, moves, count = ibp_kv_compact(table, refs, page_tokens)
    ibp_kv_copy(pages, moves, count)                        # in place
    table, lens, refs = ibp_kv_accept(pages, table, lens, refs, n_draft, path, n_accept)
    out, lse = ibp_tree_attention(q, k, v, table, lens, mask=mask)
    ibp_kv_summarize(k, table, lens, codes, scales)         # in place
    out, lse, picked = ibp_sparse_attention(q, k, v, table, lens, codes, scales, budget)
    ibp_kv_get_status()                                     # raises on a data error

Keys and values of a layer are tensors ``[n_pages, heads, page_tokens, dim]``
(bfloat16 or float16) of any strides whose last is 1: tokens-first pages are a
transposed view.  The page copies also take ``[n_pools, n_pages, heads,
page_tokens, dim]``, every layer's K and V at once.  ``table`` is int32
``[n_seqs, max_pages]``, ``lens`` int32 ``[n_seqs]``, ``refs`` int32
``[n_pages]``, all on the device.

``stream`` is a torch stream or a raw handle (default: the current stream);
results and scratch are allocated for that stream.  Data errors go to a status
word: the caller's own (``status``, an int32 device tensor) or the device's,
read by ``ibp_kv_get_status`` (call it once before the first call is captured
in a graph: it makes the word).  Nothing here has a backward pass: one that
reaches an attention call raises an error.
"""

from __future__ import annotations

import contextlib
import ctypes
import math
import threading

import torch

from . import ibp
from .ibp import IBP_OK, IbpError

IBP_KV_BF16 = 0
IBP_KV_F16 = 1
IBP_KV_MAX_DIM = 256
IBP_SPARSE_MAX_BUDGET = 4096
IBP_KV_WAIT_CYCLES = 1 << 32

_DTYPES = {torch.bfloat16: IBP_KV_BF16, torch.float16: IBP_KV_F16}


class _Pages(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pools", ctypes.c_uint64), ("pool_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_uint64), ("page_stride", ctypes.c_int64), ("heads", ctypes.c_uint32),
                ("head_stride", ctypes.c_int64), ("page_tokens", ctypes.c_uint32),
                ("token_stride", ctypes.c_int64), ("dim", ctypes.c_uint32), ("elem_bytes", ctypes.c_uint32)]


class _Seqs(ctypes.Structure):
    _fields_ = [("table", ctypes.c_void_p), ("lens", ctypes.c_void_p), ("n_seqs", ctypes.c_uint32),
                ("max_pages", ctypes.c_uint32)]


_bound = None


def _load():
    global _bound
    lib = ibp.load()
    if _bound is lib:
        return lib
    vp, u64, i64, u32, i32 = ctypes.c_void_p, ctypes.c_uint64, ctypes.c_int64, ctypes.c_uint32, ctypes.c_int
    size, f32 = ctypes.c_size_t, ctypes.c_float
    pages, seqs = ctypes.POINTER(_Pages), ctypes.POINTER(_Seqs)
    sigs = {
        "ibp_kv_fork": ([seqs, u32, vp, u64, vp, u32, vp, vp, vp, vp, vp, vp, size, vp, vp], i32),
        "ibp_kv_free": ([seqs, u32, vp, u64, vp, u32, vp, vp, vp, vp, vp], i32),
        "ibp_kv_compact": ([seqs, u32, vp, u64, vp, vp, vp, vp, vp, size, vp, vp], i32),
        "ibp_kv_pages_workspace": ([u64, u32], size),
        "ibp_kv_copy": ([pages, vp, vp, u32, vp, vp], i32),
        "ibp_kv_accept": ([pages, seqs, vp, vp, vp, vp, u32, vp, vp, vp, vp, vp], i32),
        "ibp_tree_attention": ([pages, pages, u32, seqs, vp, i64, i64, i64, u32, u32, vp, vp, f32, vp, vp, vp, size,
                                vp, vp], i32),
        "ibp_tree_attention_workspace": ([u32] * 7, size),
        "ibp_kv_set_wait_limit": ([u64], u64),
        "ibp_kv_summarize": ([pages, u32, seqs, vp, vp, vp, vp, vp], i32),
        "ibp_sparse_attention": ([pages, pages, u32, seqs, vp, vp, vp, i64, i64, i64, u32, u32, vp, u32, u32, u32,
                                  f32, vp, vp, vp, vp, size, vp, vp], i32),
        "ibp_sparse_attention_workspace": ([u32] * 8, size),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _bound = lib
    return lib


# ---------------------------------------------------------------------------
# Arguments
#
# A call's checks depend on its tensors' shapes, strides, types and devices alone.
# They run once for each combination of these, with the tensors' device current (the
# scratch goes by its number of SMs); what they yield (the C structures without
# their addresses, sizes of results and scratch) is kept per thread under that
# combination, and a call fills in its addresses.  Nothing of a call's data or
# addresses is kept.


class _Checked(threading.local):
    def __init__(self):
        self.calls = {}


_checked = _Checked()
_MOST_CHECKED = 1024


def _form(t: torch.Tensor | None):
    """What the checks look at."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _once(key, check):
    calls = _checked.calls
    found = calls.get(key)
    if found is None:
        found = check()
        if len(calls) >= _MOST_CHECKED:
            calls.clear()
        calls[key] = found
    return found


def _ints(name: str, t: torch.Tensor, *shape):
    """shape: the wanted sizes, None where any will do."""
    if t.dtype != torch.int32 or not t.is_contiguous() or t.dim() != len(shape):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {len(shape)} dimension(s)")
    if any(want is not None and have != want for have, want in zip(t.shape, shape)):
        raise ValueError(f"{name} is {list(t.shape)}, not {[w if w is not None else 'any' for w in shape]}")


def _on_device(name: str, t: torch.Tensor):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")


def _sequences(table: torch.Tensor, lens: torch.Tensor) -> _Seqs:
    _ints("table", table, None, None)
    _ints("lens", lens, table.shape[0])
    return _Seqs(0, 0, table.shape[0], table.shape[1])


def _as_pages(name: str, t: torch.Tensor, pools: bool = False) -> _Pages:
    _on_device(name, t)
    if pools and t.dim() == 5:
        n_pools, shape, strides = t.shape[0], t.shape[1:], t.stride()
        pool_stride, strides = strides[0], strides[1:]
    elif t.dim() == 4:
        n_pools, pool_stride, shape, strides = 1, 0, t.shape, t.stride()
    else:
        raise ValueError(f"{name} must have the dimensions {'[pools,] ' if pools else ''}pages, heads, tokens, dim")
    if shape[3] > 1 and strides[3] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return _Pages(0, n_pools, pool_stride, shape[0], strides[0], shape[1], strides[1], shape[2], strides[2],
                  shape[3], t.element_size())


def _dtype(*tensors: torch.Tensor) -> int:
    dt = tensors[0].dtype
    if dt not in _DTYPES or any(t.dtype != dt for t in tensors):
        raise ValueError("queries, keys and values must all be bfloat16 or all float16")
    return _DTYPES[dt]


def _given(name: str, t: torch.Tensor, shape, dtype) -> torch.Tensor:
    """A result tensor of the caller's."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}")
    return t


def _scratch(workspace: torch.Tensor | None, size: int, device: torch.device) -> torch.Tensor | None:
    if workspace is None:
        return torch.empty(size, dtype=torch.uint8, device=device) if size else None
    if workspace.numel() * workspace.element_size() < size or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous and hold {size} bytes")
    return workspace


_as_is = contextlib.nullcontext()


def _for(stream, device: torch.device):
    """(stream handle, context in which results of that stream are allocated)."""
    index = device.index
    if index is None:
        raise ValueError("pages and tables must be on a CUDA device")
    if stream is None:
        handle = ibp._raw_stream(index) if ibp._raw_stream is not None else ibp._stream(None, device)
        return handle, _as_is if index == torch.cuda.current_device() else torch.cuda.device(device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    return stream.cuda_stream, torch.cuda.stream(stream)


# ---------------------------------------------------------------------------
# Status

_status_words: dict[int, torch.Tensor] = {}


def _status_word(index: int) -> torch.Tensor:
    word = _status_words.get(index)
    if word is None:
        if torch.cuda.is_current_stream_capturing():
            raise RuntimeError("the device's status word is not made yet, which a capture cannot hold: call "
                               "ibp_kv_get_status() before it, or pass a status word")
        with torch.cuda.device(index):
            word = torch.zeros(1, dtype=torch.int32, device="cuda")
            torch.cuda.synchronize()  # made once: every stream may use it
        word = _status_words.setdefault(index, word)
    return word


def _status(status: torch.Tensor | None, device: torch.device) -> int:
    if status is None:
        word = _status_words.get(device.index)
        return (_status_word(device.index) if word is None else word).data_ptr()
    if status.element_size() != 4 or status.numel() < 1:
        raise ValueError("status must be a 32-bit word")
    return status.data_ptr()


def ibp_kv_get_status(device: int | None = None, raise_on_error: bool = True) -> int:
    """Waits for the device, returns the first data error of the calls that
    named no status word of their own since the last call, and clears it.  The
    first use of a device makes its word, which a graph capture cannot hold: a
    program that captures its first call calls this before."""
    device = torch.cuda.current_device() if device is None else int(device)
    word = _status_word(device)
    torch.cuda.synchronize(device)
    code = int(word.item())
    if code != IBP_OK:
        word.zero_()
        torch.cuda.synchronize(device)
        if raise_on_error:
            raise IbpError(code, "ibp_kv_get_status")
    return code


def _check(code: int, where: str):
    if code != IBP_OK:
        raise IbpError(code, where)


# ---------------------------------------------------------------------------
# Pages


def ibp_kv_fork(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, parents: torch.Tensor,
                page_tokens: int, status: torch.Tensor | None = None, stream=None):
    """The next batch: row i continues row parents[i].  Returns new (table,
    lens, refs) and the page copies to make, (moves, count) for ibp_kv_copy."""
    lib = _load()

    def check():
        _on_device("table", table)
        _ints("refs", refs, None)
        _ints("parents", parents, None)
        n_pages, n_out = refs.shape[0], parents.shape[0]
        return _sequences(table, lens), n_pages, n_out, lib.ibp_kv_pages_workspace(n_pages, n_out)

    key = ("fork", _form(table), _form(lens), _form(refs), _form(parents))
    device = table.device
    handle, where = _for(stream, device)
    with where:
        seqs, n_pages, n_out, size = _once(key, check)
        table_out = torch.empty((n_out, table.shape[1]), dtype=torch.int32, device=device)
        lens_out = torch.empty(n_out, dtype=torch.int32, device=device)
        refs_out = torch.empty(n_pages, dtype=torch.int32, device=device)
        moves = torch.empty((n_out, 3), dtype=torch.int32, device=device)
        count = torch.empty(1, dtype=torch.int32, device=device)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv_fork(seqs, page_tokens, refs.data_ptr(), n_pages, parents.data_ptr(), n_out,
                               table_out.data_ptr(), lens_out.data_ptr(), refs_out.data_ptr(), moves.data_ptr(),
                               count.data_ptr(), ws.data_ptr(), size, _status(status, device), handle),
               "ibp_kv_fork")
    return table_out, lens_out, refs_out, moves, count


def ibp_kv_free(table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor, seqs: torch.Tensor, page_tokens: int,
                inplace: bool = False, status: torch.Tensor | None = None, stream=None):
    """Frees the listed sequences; returns (table, lens, refs), the arguments
    themselves with `inplace`."""
    lib = _load()

    def check():
        _on_device("table", table)
        _ints("refs", refs, None)
        _ints("seqs", seqs, None)
        return _sequences(table, lens), refs.shape[0], seqs.shape[0]

    device = table.device
    handle, where = _for(stream, device)
    with where:
        s, n_pages, n_rows = _once(("free", _form(table), _form(lens), _form(refs), _form(seqs)), check)
        out = (table, lens, refs)
        if not inplace:
            out = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
        s.table, s.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv_free(s, page_tokens, refs.data_ptr(), n_pages, seqs.data_ptr(), n_rows,
                               out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), _status(status, device),
                               handle), "ibp_kv_free")
    return out


def ibp_kv_compact(table: torch.Tensor, refs: torch.Tensor, page_tokens: int, inplace: bool = False,
                   status: torch.Tensor | None = None, stream=None):
    """Live pages to the front of the pool; returns (table, refs, moves, count),
    the first two the arguments themselves with `inplace`."""
    lib = _load()

    def check():
        _on_device("table", table)
        _ints("table", table, None, None)
        _ints("refs", refs, None)
        n_pages = refs.shape[0]
        return _Seqs(0, 0, *table.shape), n_pages, lib.ibp_kv_pages_workspace(n_pages, 0)

    device = table.device
    handle, where = _for(stream, device)
    with where:
        seqs, n_pages, size = _once(("compact", _form(table), _form(refs)), check)
        out = (table, refs) if inplace else (torch.empty_like(table), torch.empty_like(refs))
        moves = torch.empty((n_pages, 3), dtype=torch.int32, device=device)
        count = torch.empty(1, dtype=torch.int32, device=device)
        ws = torch.empty(size, dtype=torch.uint8, device=device)
        seqs.table = table.data_ptr()  # the lengths are not read: the references say which pages live
        _check(lib.ibp_kv_compact(seqs, page_tokens, refs.data_ptr(), n_pages, out[0].data_ptr(), out[1].data_ptr(),
                                  moves.data_ptr(), count.data_ptr(), ws.data_ptr(), size, _status(status, device),
                                  handle), "ibp_kv_compact")
    return *out, moves, count


def ibp_kv_copy(pages: torch.Tensor, moves: torch.Tensor, count: torch.Tensor, status: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """Copies pages as `moves` lists them, in place and in every pool."""
    lib = _load()

    def check():
        _ints("moves", moves, None, 3)
        _ints("count", count, 1)
        return _as_pages("pages", pages, pools=True), moves.shape[0]

    device = pages.device
    handle, where = _for(stream, device)
    with where:
        p, most = _once(("copy", _form(pages), _form(moves), _form(count)), check)
        p.data = pages.data_ptr()
        _check(lib.ibp_kv_copy(p, moves.data_ptr(), count.data_ptr(), most, _status(status, device), handle),
               "ibp_kv_copy")
    return pages


def ibp_kv_accept(pages: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, refs: torch.Tensor,
                  n_draft: torch.Tensor, path: torch.Tensor, n_accept: torch.Tensor, inplace: bool = False,
                  status: torch.Tensor | None = None, stream=None):
    """Keeps the accepted tokens of each sequence's draft (its last n_draft[b]
    tokens): path[b][: n_accept[b]] move to the draft's front in every pool.
    Returns (table, lens, refs)."""
    lib = _load()

    def check():
        p, n = _as_pages("pages", pages, pools=True), table.shape[0]
        _ints("refs", refs, p.n_pages)
        _ints("n_draft", n_draft, n)
        _ints("path", path, n, None)
        _ints("n_accept", n_accept, n)
        return p, _sequences(table, lens), path.shape[1]

    key = ("accept", _form(pages), _form(table), _form(lens), _form(refs), _form(n_draft), _form(path),
           _form(n_accept))
    device = pages.device
    handle, where = _for(stream, device)
    with where:
        p, seqs, most = _once(key, check)
        out = (table, lens, refs)
        if seqs.n_seqs == 0:
            return out if inplace else (table.clone(), lens.clone(), refs.clone())
        if not inplace:
            out = torch.empty_like(table), torch.empty_like(lens), torch.empty_like(refs)
        p.data = pages.data_ptr()
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv_accept(p, seqs, refs.data_ptr(), n_draft.data_ptr(), path.data_ptr(), n_accept.data_ptr(),
                                 most, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(),
                                 _status(status, device), handle), "ibp_kv_accept")
    return out


# ---------------------------------------------------------------------------
# Attention


class _NoBackward(torch.autograd.Function):
    """Passes results on; a gradient that comes back for them is an error, not silence."""

    @staticmethod
    def forward(ctx, name, out, lse, *inputs):
        ctx.name = name
        return out.view_as(out), lse.view_as(lse)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no backward pass: detach q, k and v, or call it under torch.no_grad()")


def _results(name: str, out: torch.Tensor, lse: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor):
    if (q.requires_grad or k.requires_grad or v.requires_grad) and torch.is_grad_enabled():
        return _NoBackward.apply(name, out, lse, q, k, v)
    return out, lse


def _heads(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor):
    """(k pages, v pages, dtype, sequences) of an attention call."""
    kp, vp = _as_pages("k", k), _as_pages("v", v)
    seqs = _sequences(table, lens)
    _on_device("q", q)
    if q.dim() != 4 or q.shape[0] != seqs.n_seqs or q.shape[3] != kp.dim:
        raise ValueError("q must be [n_seqs, T, q_heads, dim] with the table's sequences and the pages' dim")
    if q.shape[3] > 1 and q.stride(3) != 1:
        raise ValueError("the last dimension of q must be contiguous")
    return kp, vp, _dtype(k, v, q), seqs


def ibp_tree_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                       mask: torch.Tensor | None = None, n_draft: torch.Tensor | None = None,
                       scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Attention of each sequence's draft, its last T (or n_draft[b]) tokens.

    mask   int32 [n_seqs, T, ceil(T / 32)]: bit i of row t lets drafted token t
           see drafted token i; None: a chain (i <= t).
    scale  default 1 / sqrt(dim).
    Returns (out [n_seqs, T, q_heads, dim], lse [n_seqs, T, q_heads])."""
    lib = _load()

    def check():
        kp, vp, dt, seqs = _heads(q, k, v, table, lens)
        T, heads = q.shape[1], q.shape[2]
        if mask is not None:
            _ints("mask", mask, seqs.n_seqs, T, (T + 31) // 32)
        if n_draft is not None:
            _ints("n_draft", n_draft, seqs.n_seqs)
        size = lib.ibp_tree_attention_workspace(seqs.n_seqs, seqs.max_pages, kp.page_tokens, T, heads, kp.heads, kp.dim)
        return kp, vp, dt, seqs, (*q.stride()[:3], T, heads), size, 1.0 / math.sqrt(kp.dim)

    key = ("tree", _form(q), _form(k), _form(v), _form(table), _form(lens), _form(mask), _form(n_draft))
    device = k.device
    handle, where = _for(stream, device)
    with where:
        kp, vp, dt, seqs, rows, size, usual = _once(key, check)
        out = torch.empty(q.shape, dtype=q.dtype, device=device) if out is None else _given("out", out, q.shape, q.dtype)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=device)
        else:
            _given("lse", lse, q.shape[:3], torch.float32)
        ws = _scratch(workspace, size, device)
        kp.data, vp.data = k.data_ptr(), v.data_ptr()
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_tree_attention(kp, vp, dt, seqs, q.data_ptr(), *rows,
                                      None if n_draft is None else n_draft.data_ptr(),
                                      None if mask is None else mask.data_ptr(), usual if scale is None else scale,
                                      out.data_ptr(), lse.data_ptr(), None if ws is None else ws.data_ptr(), size,
                                      _status(status, device), handle), "ibp_tree_attention")
    return _results("ibp_tree_attention", out, lse, q, k, v)


def ibp_kv_set_wait_limit(cycles: int = IBP_KV_WAIT_CYCLES) -> int:
    """Clock cycles after which a wait inside ibp_tree_attention gives up with
    IBP_ETIMEOUT (0: at once, to test what follows); returns the limit before."""
    return _load().ibp_kv_set_wait_limit(cycles)


def _bounds(k: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor):
    n_pages, heads, _, dim = k.shape
    _given("codes", codes, (n_pages, heads, 2, dim), torch.int8)
    _given("scales", scales, (n_pages, heads), torch.float32)


def ibp_kv_summarize(k: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, codes: torch.Tensor,
                     scales: torch.Tensor, first: torch.Tensor | None = None, status: torch.Tensor | None = None,
                     stream=None):
    """8-bit bounds of the keys of every page that holds a position from
    first[b] on (None: every page), into codes [n_pages, heads, 2, dim] int8
    and scales [n_pages, heads] float32.  Returns (codes, scales)."""
    lib = _load()

    def check():
        kp, seqs = _as_pages("k", k), _sequences(table, lens)
        _bounds(k, codes, scales)
        if first is not None:
            _ints("first", first, seqs.n_seqs)
        return kp, seqs, _dtype(k)

    key = ("summarize", _form(k), _form(table), _form(lens), _form(codes), _form(scales), _form(first))
    device = k.device
    handle, where = _for(stream, device)
    with where:
        kp, seqs, dt = _once(key, check)
        kp.data = k.data_ptr()
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv_summarize(kp, dt, seqs, None if first is None else first.data_ptr(), codes.data_ptr(),
                                    scales.data_ptr(), _status(status, device), handle), "ibp_kv_summarize")
    return codes, scales


def ibp_sparse_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, lens: torch.Tensor,
                         codes: torch.Tensor, scales: torch.Tensor, budget: int, keep_first: int = 1,
                         keep_last: int = 1, n_query: torch.Tensor | None = None, scale: float | None = None,
                         out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                         pages: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         status: torch.Tensor | None = None, stream=None):
    """Attention of each sequence's last T (or n_query[b]) tokens over `budget`
    pages per query and kv head, selected by the bounds of ibp_kv_summarize;
    the first keep_first and the last keep_last pages are always among them.

    Returns (out, lse, pages): pages int32 [n_seqs, T, kv_heads, budget], the
    selected places in the table row ascending, then -1."""
    lib = _load()

    def check():
        kp, vp, dt, seqs = _heads(q, k, v, table, lens)
        T, heads = q.shape[1], q.shape[2]
        _bounds(k, codes, scales)
        if not 1 <= budget <= IBP_SPARSE_MAX_BUDGET or keep_first < 0 or keep_last < 1 or keep_first + keep_last > budget:
            raise ValueError("budget must hold keep_first >= 0 and keep_last >= 1 pages and be at most "
                             f"{IBP_SPARSE_MAX_BUDGET}")
        if n_query is not None:
            _ints("n_query", n_query, seqs.n_seqs)
        size = lib.ibp_sparse_attention_workspace(seqs.n_seqs, seqs.max_pages, kp.page_tokens, T, heads, kp.heads, kp.dim,
                                                  budget)
        return kp, vp, dt, seqs, (*q.stride()[:3], T, heads), size, 1.0 / math.sqrt(kp.dim)

    key = ("sparse", _form(q), _form(k), _form(v), _form(table), _form(lens), _form(codes), _form(scales),
           _form(n_query), budget, keep_first, keep_last)
    device = k.device
    handle, where = _for(stream, device)
    with where:
        kp, vp, dt, seqs, rows, size, usual = _once(key, check)
        out = torch.empty(q.shape, dtype=q.dtype, device=device) if out is None else _given("out", out, q.shape, q.dtype)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=device)
        else:
            _given("lse", lse, q.shape[:3], torch.float32)
        wanted = (seqs.n_seqs, rows[3], kp.heads, budget)
        if pages is None:
            pages = torch.empty(wanted, dtype=torch.int32, device=device)
        else:
            _given("pages", pages, wanted, torch.int32)
        ws = _scratch(workspace, size, device)
        kp.data, vp.data = k.data_ptr(), v.data_ptr()
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_sparse_attention(kp, vp, dt, seqs, codes.data_ptr(), scales.data_ptr(), q.data_ptr(), *rows,
                                        None if n_query is None else n_query.data_ptr(), budget, keep_first,
                                        keep_last, usual if scale is None else scale, out.data_ptr(), lse.data_ptr(),
                                        pages.data_ptr(), None if ws is None else ws.data_ptr(), size,
                                        _status(status, device), handle), "ibp_sparse_attention")
    return *_results("ibp_sparse_attention", out, lse, q, k, v), pages
