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
    ibp_kv4_store(k, v, k4, v4, table, lens)                # into a cache in 4 bits, in place
    k, v = ibp_kv4_load(k4, v4, table, lens, n)             # the last n tokens, as it holds them
    out, lse = ibp_kv4_attention(q, k4, v4, table, lens, mask=mask)
    path, n_accept, token = ibp_kv_verify(p, tokens, u, q=draft, parents=parents)
    weights = ibp_kv_weigh(q, k, table, lens, lse, weights) # k: pages of 16 bits, or a cache in 4 bits
    path, n_draft, n_keep, weights = ibp_kv_evict(weights, lens, budget)
    ibp_kv_get_status()                                     # raises on a data error

Keys and values of a layer are tensors ``[n_pages, heads, page_tokens, dim]``
(bfloat16 or float16) of any strides whose last is 1: tokens-first pages are a
transposed view.  The page copies also take ``[n_pools, n_pages, heads,
page_tokens, dim]``, every layer's K and V at once.  A cache in 4 bits is a pair
``(codes, scales)``: uint8 ``[n_pages, heads, page_tokens, dim / 2]`` and the queries'
type ``[n_pages, heads, page_tokens, dim / 32]``; to the page copies either is a pool.
``table`` is int32 ``[n_seqs, max_pages]``, ``lens`` int32 ``[n_seqs]``, ``refs`` int32
``[n_pages]``, all on the device.

``stream`` is a torch stream or a raw handle (default: the current stream);
results and scratch are allocated for that stream.  Data errors go to a status
word: the caller's own (``status``, an int32 device tensor) or the device's,
read by ``ibp_kv_get_status`` (call it once before the first call is captured
in a graph: it makes the word).  Nothing here has a backward pass: one that
reaches an attention call, loaded keys and values or accumulated weights raises an
error.
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
IBP_KV4_GROUP = 32
IBP_VERIFY_MAX_VOCAB = 262144
IBP_VERIFY_MAX_DRAFT = 1024

_DTYPES = {torch.bfloat16: IBP_KV_BF16, torch.float16: IBP_KV_F16}


class _Pages(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("n_pools", ctypes.c_uint64), ("pool_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_uint64), ("page_stride", ctypes.c_int64), ("heads", ctypes.c_uint32),
                ("head_stride", ctypes.c_int64), ("page_tokens", ctypes.c_uint32),
                ("token_stride", ctypes.c_int64), ("dim", ctypes.c_uint32), ("elem_bytes", ctypes.c_uint32)]


class _Pages4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("scales", ctypes.c_void_p), ("scale_page_stride", ctypes.c_int64),
                ("scale_head_stride", ctypes.c_int64), ("scale_token_stride", ctypes.c_int64),
                ("n_pages", ctypes.c_uint64), ("heads", ctypes.c_uint32), ("page_tokens", ctypes.c_uint32),
                ("dim", ctypes.c_uint32)]


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
    pages, seqs, pages4 = ctypes.POINTER(_Pages), ctypes.POINTER(_Seqs), ctypes.POINTER(_Pages4)
    weigh = [u32, seqs, vp, i64, i64, i64, u32, u32, vp, vp, f32, vp, vp, vp, u32, f32, vp, vp]
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
        "ibp_kv4_store": ([pages4, pages4, u32, seqs, vp, i64, i64, i64, vp, i64, i64, i64, u32, vp, vp, vp], i32),
        "ibp_kv4_load": ([pages4, pages4, u32, seqs, u32, vp, vp, vp, vp, vp], i32),
        "ibp_kv4_attention": ([pages4, pages4, u32, seqs, vp, i64, i64, i64, u32, u32, vp, vp, f32, vp, vp, vp, size,
                               vp, vp], i32),
        "ibp_kv4_attention_workspace": ([u32] * 7, size),
        "ibp_kv_verify": ([vp, i64, i64, vp, i64, i64, u32, vp, vp, vp, u32, u32, vp, vp, vp, vp, vp, vp], i32),
        "ibp_kv_weigh": ([pages, *weigh], i32),
        "ibp_kv4_weigh": ([pages4, *weigh], i32),
        "ibp_kv_evict": ([vp, u32, vp, u32, u32, u32, u32, vp, vp, vp, vp, vp, vp], i32),
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
    tokens): path[b][: n_accept[b]] move to the draft's front in every pool.  A
    sequence with a page of several references among those that tokens move onto is
    left alone (status IBP_EINVAL).  Returns (table, lens, refs)."""
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


class _NoBackwardOfOne(torch.autograd.Function):
    """The same for a single result."""

    @staticmethod
    def forward(ctx, name, out, *inputs):
        ctx.name = name
        return out.view_as(out)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError(f"{ctx.name} has no backward pass: detach its inputs, or call it under torch.no_grad()")


def _result(name: str, out: torch.Tensor, *inputs: torch.Tensor):
    for t in inputs:
        if t.requires_grad and torch.is_grad_enabled():
            return _NoBackwardOfOne.apply(name, out, *inputs)
    return out


def _no_gradients(name: str, *inputs: torch.Tensor):
    """For calls that write into tensors of the caller's, which cannot carry the error to a backward."""
    if torch.is_grad_enabled() and any(t.requires_grad for t in inputs):
        raise ValueError(f"{name}: what is written in place carries no gradient: detach its inputs, or call it "
                         "under torch.no_grad()")


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


# ---------------------------------------------------------------------------
# Caches in 4 bits


def _form4(pages):
    return _form(pages[0]), _form(pages[1])


def _as_pages4(name: str, pages) -> _Pages4:
    codes, scales = pages
    for what, t in (("codes", codes), ("scales", scales)):
        _on_device(f"the {what} of {name}", t)
        if t.dim() != 4 or (t.shape[3] > 1 and t.stride(3) != 1):
            raise ValueError(f"the {what} of {name} must have the dimensions pages, heads, tokens, dim, the last contiguous")
    if codes.dtype != torch.uint8 or scales.dtype not in _DTYPES:
        raise ValueError(f"{name} must be codes in uint8 and scales in bfloat16 or float16")
    dim = 2 * codes.shape[3]
    if dim % IBP_KV4_GROUP or scales.shape != (*codes.shape[:3], dim // IBP_KV4_GROUP) or codes.device != scales.device:
        raise ValueError(f"the scales of {name} must be one for each {IBP_KV4_GROUP} elements of the codes, on their device")
    return _Pages4(0, *codes.stride()[:3], 0, *scales.stride()[:3], *codes.shape[:3], dim)


def _place4(p: _Pages4, pages):
    p.codes, p.scales = pages[0].data_ptr(), pages[1].data_ptr()


def _caches4(k4, v4, table: torch.Tensor, lens: torch.Tensor):
    kp, vp = _as_pages4("k4", k4), _as_pages4("v4", v4)
    return kp, vp, _dtype(k4[1], v4[1]), _sequences(table, lens)


def ibp_kv4_store(k: torch.Tensor, v: torch.Tensor, k4, v4, table: torch.Tensor, lens: torch.Tensor,
                  n_new: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """Puts k and v [n_seqs, T, heads, dim], the last T (or n_new[b]) tokens of each
    sequence, into caches in 4 bits, (codes, scales) each, in place.  Returns (k4, v4).
    The cache carries no gradient: tensors that require one are refused where gradients are
    enabled."""
    lib = _load()
    _no_gradients("ibp_kv4_store", k, v, k4[1], v4[1])

    def check():
        kp, vp, dt, seqs = _caches4(k4, v4, table, lens)
        for name, t in (("k", k), ("v", v)):
            _on_device(name, t)
            if t.dim() != 4 or t.shape != (seqs.n_seqs, k.shape[1], kp.heads, kp.dim) or t.dtype != k4[1].dtype:
                raise ValueError(f"{name} must be [n_seqs, T, heads, dim] of the cache's type")
            if t.stride(3) != 1:
                raise ValueError(f"the last dimension of {name} must be contiguous")
        if n_new is not None:
            _ints("n_new", n_new, seqs.n_seqs)
        return kp, vp, dt, seqs, k.stride()[:3], v.stride()[:3]

    key = ("store4", _form(k), _form(v), _form4(k4), _form4(v4), _form(table), _form(lens), _form(n_new))
    device = k4[0].device
    handle, where = _for(stream, device)
    with where:
        kp, vp, dt, seqs, ks, vs = _once(key, check)
        _place4(kp, k4), _place4(vp, v4)
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv4_store(kp, vp, dt, seqs, k.data_ptr(), *ks, v.data_ptr(), *vs, k.shape[1],
                                 None if n_new is None else n_new.data_ptr(), _status(status, device), handle),
               "ibp_kv4_store")
    return k4, v4


def ibp_kv4_load(k4, v4, table: torch.Tensor, lens: torch.Tensor, T: int, n_load: torch.Tensor | None = None,
                 k: torch.Tensor | None = None, v: torch.Tensor | None = None, status: torch.Tensor | None = None,
                 stream=None):
    """The last T (or n_load[b]) tokens of each sequence as caches in 4 bits hold them:
    (k, v) [n_seqs, T, heads, dim], zeros behind n_load[b]."""
    lib = _load()

    def check():
        kp, vp, dt, seqs = _caches4(k4, v4, table, lens)
        if n_load is not None:
            _ints("n_load", n_load, seqs.n_seqs)
        return kp, vp, dt, seqs

    device = k4[0].device
    handle, where = _for(stream, device)
    with where:
        kp, vp, dt, seqs = _once(("load4", _form4(k4), _form4(v4), _form(table), _form(lens), _form(n_load)), check)
        shape = seqs.n_seqs, T, kp.heads, kp.dim
        k = torch.empty(shape, dtype=k4[1].dtype, device=device) if k is None else _given("k", k, shape, k4[1].dtype)
        v = torch.empty(shape, dtype=k4[1].dtype, device=device) if v is None else _given("v", v, shape, k4[1].dtype)
        _place4(kp, k4), _place4(vp, v4)
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv4_load(kp, vp, dt, seqs, T, None if n_load is None else n_load.data_ptr(), k.data_ptr(),
                                v.data_ptr(), _status(status, device), handle), "ibp_kv4_load")
    return _results("ibp_kv4_load", k, v, k4[1], v4[1], v4[1])


def _queries(q: torch.Tensor, seqs: _Seqs, dim: int, dtype, mask, n_draft):
    _on_device("q", q)
    if q.dim() != 4 or q.shape[0] != seqs.n_seqs or q.shape[3] != dim or q.dtype != dtype:
        raise ValueError("q must be [n_seqs, T, q_heads, dim] with the table's sequences and the cache's dim and type")
    if q.shape[3] > 1 and q.stride(3) != 1:
        raise ValueError("the last dimension of q must be contiguous")
    T = q.shape[1]
    if mask is not None:
        _ints("mask", mask, seqs.n_seqs, T, (T + 31) // 32)
    if n_draft is not None:
        _ints("n_draft", n_draft, seqs.n_seqs)
    return *q.stride()[:3], T, q.shape[2]


def ibp_kv4_attention(q: torch.Tensor, k4, v4, table: torch.Tensor, lens: torch.Tensor,
                      mask: torch.Tensor | None = None, n_draft: torch.Tensor | None = None,
                      scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                      workspace: torch.Tensor | None = None, status: torch.Tensor | None = None, stream=None):
    """ibp_tree_attention over caches in 4 bits, (codes, scales) each.
    Returns (out [n_seqs, T, q_heads, dim], lse [n_seqs, T, q_heads])."""
    lib = _load()

    def check():
        kp, vp, dt, seqs = _caches4(k4, v4, table, lens)
        rows = _queries(q, seqs, kp.dim, k4[1].dtype, mask, n_draft)
        size = lib.ibp_kv4_attention_workspace(seqs.n_seqs, seqs.max_pages, kp.page_tokens, *rows[3:], kp.heads, kp.dim)
        return kp, vp, dt, seqs, rows, size, 1.0 / math.sqrt(kp.dim)

    key = ("attention4", _form(q), _form4(k4), _form4(v4), _form(table), _form(lens), _form(mask), _form(n_draft))
    device = k4[0].device
    handle, where = _for(stream, device)
    with where:
        kp, vp, dt, seqs, rows, size, usual = _once(key, check)
        out = torch.empty(q.shape, dtype=q.dtype, device=device) if out is None else _given("out", out, q.shape, q.dtype)
        if lse is None:
            lse = torch.empty(q.shape[:3], dtype=torch.float32, device=device)
        else:
            _given("lse", lse, q.shape[:3], torch.float32)
        ws = _scratch(workspace, size, device)
        _place4(kp, k4), _place4(vp, v4)
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        _check(lib.ibp_kv4_attention(kp, vp, dt, seqs, q.data_ptr(), *rows,
                                     None if n_draft is None else n_draft.data_ptr(),
                                     None if mask is None else mask.data_ptr(), usual if scale is None else scale,
                                     out.data_ptr(), lse.data_ptr(), None if ws is None else ws.data_ptr(), size,
                                     _status(status, device), handle), "ibp_kv4_attention")
    return _results("ibp_kv4_attention", out, lse, q, k4[1], v4[1])


# ---------------------------------------------------------------------------
# Drafted tokens, eviction


def _floats(name: str, t: torch.Tensor, *shape):
    """shape: the wanted sizes, None where any will do."""
    _on_device(name, t)
    if (t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != len(shape)
            or any(want is not None and have != want for have, want in zip(t.shape, shape))):
        raise ValueError(f"{name} must be a contiguous float32 tensor of shape {[w if w is not None else 'any' for w in shape]}")


def _probabilities(name: str, t: torch.Tensor, *shape):
    _on_device(name, t)
    if t.dtype != torch.float32 or t.shape != shape or (t.shape[2] > 1 and t.stride(2) != 1):
        raise ValueError(f"{name} must be a float32 tensor of shape {list(shape)}, the last dimension contiguous")


def ibp_kv_verify(p: torch.Tensor, tokens: torch.Tensor, u: torch.Tensor, q: torch.Tensor | None = None,
                  parents: torch.Tensor | None = None, n_draft: torch.Tensor | None = None,
                  status: torch.Tensor | None = None, stream=None):
    """Drafted tokens against the target's probabilities, and the next token.

    p        float32 [n_seqs, T + 1, vocab]: row 0 behind the context, row 1 + t
             behind drafted token t.
    tokens   int32 [n_seqs, T].
    u        float32 [n_seqs, T + 1], uniform in [0, 1): u[:, t] decides on token t,
             the last column draws.
    q        float32 [n_seqs, T, vocab], what the draft drew from (row 1 + parents of a
             token); None: every drafted token was certain.
    parents  int32 [n_seqs, T], an earlier token or -1; None: a chain.
    Returns (path [n_seqs, T], n_accept [n_seqs], token [n_seqs]), the first two as
    ibp_kv_accept takes them."""
    lib = _load()

    def check():
        _on_device("tokens", tokens)
        _ints("tokens", tokens, None, None)
        n, T = tokens.shape
        if p.dim() != 3:
            raise ValueError("p must have the dimensions sequences, tokens + 1, vocabulary")
        V = p.shape[2]
        _probabilities("p", p, n, T + 1, V)
        _floats("u", u, n, T + 1)
        if q is not None:
            _probabilities("q", q, n, T, V)
        if parents is not None:
            _ints("parents", parents, n, T)
        if n_draft is not None:
            _ints("n_draft", n_draft, n)
        if not 1 <= V <= IBP_VERIFY_MAX_VOCAB or T > IBP_VERIFY_MAX_DRAFT:
            raise ValueError(f"a vocabulary of 1 to {IBP_VERIFY_MAX_VOCAB} and at most {IBP_VERIFY_MAX_DRAFT} drafted tokens")
        return n, T, V, p.stride()[:2], (0, 0) if q is None else q.stride()[:2]

    key = ("verify", _form(p), _form(tokens), _form(u), _form(q), _form(parents), _form(n_draft))
    device = p.device
    handle, where = _for(stream, device)
    with where:
        n, T, V, ps, qs = _once(key, check)
        path = torch.empty((n, T), dtype=torch.int32, device=device)
        n_accept = torch.empty(n, dtype=torch.int32, device=device)
        token = torch.empty(n, dtype=torch.int32, device=device)
        _check(lib.ibp_kv_verify(p.data_ptr(), *ps, None if q is None else q.data_ptr(), *qs, V, tokens.data_ptr(),
                                 None if parents is None else parents.data_ptr(),
                                 None if n_draft is None else n_draft.data_ptr(), n, T, u.data_ptr(), path.data_ptr(),
                                 n_accept.data_ptr(), token.data_ptr(), _status(status, device), handle), "ibp_kv_verify")
    return path, n_accept, token


def ibp_kv_weigh(q: torch.Tensor, k, table: torch.Tensor, lens: torch.Tensor, lse: torch.Tensor, weights: torch.Tensor,
                 mask: torch.Tensor | None = None, n_draft: torch.Tensor | None = None, scale: float | None = None,
                 decay: float = 1.0, inplace: bool = False, status: torch.Tensor | None = None, stream=None):
    """Adds the attention weight that the last T (or n_draft[b]) tokens' queries give to
    each cached position, with the lse that their attention has returned.

    k        pages of 16 bits, or a cache in 4 bits (codes, scales).
    weights  float32 [n_seqs, width], width at least the longest length.
    Returns the new weights; with `inplace` these are `weights` itself, and tensors that
    require a gradient are refused where gradients are enabled."""
    lib = _load()
    four = isinstance(k, (tuple, list))

    def check():
        kp = _as_pages4("k", k) if four else _as_pages("k", k)
        seqs = _sequences(table, lens)
        kind = k[1] if four else k
        rows = _queries(q, seqs, kp.dim, kind.dtype, mask, n_draft)
        _floats("lse", lse, *q.shape[:3])
        _floats("weights", weights, seqs.n_seqs, None)
        return kp, _dtype(kind), seqs, rows, weights.shape[1], 1.0 / math.sqrt(kp.dim)

    if inplace:
        _no_gradients("ibp_kv_weigh", q, k[1] if four else k, lse, weights)
    key = ("weigh", _form(q), _form4(k) if four else _form(k), _form(table), _form(lens), _form(lse), _form(weights),
           _form(mask), _form(n_draft))
    device = lse.device
    handle, where = _for(stream, device)
    with where:
        kp, dt, seqs, rows, width, usual = _once(key, check)
        out = weights if inplace else torch.empty_like(weights)
        if four:
            _place4(kp, k)
        else:
            kp.data = k.data_ptr()
        seqs.table, seqs.lens = table.data_ptr(), lens.data_ptr()
        call = lib.ibp_kv4_weigh if four else lib.ibp_kv_weigh
        _check(call(kp, dt, seqs, q.data_ptr(), *rows, None if n_draft is None else n_draft.data_ptr(),
                    None if mask is None else mask.data_ptr(), usual if scale is None else scale, lse.data_ptr(),
                    weights.data_ptr(), out.data_ptr(), width, decay, _status(status, device), handle), "ibp_kv_weigh")
    return _result("ibp_kv_weigh", out, q, k[1] if four else k, lse, weights)


def ibp_kv_evict(weights: torch.Tensor, lens: torch.Tensor, budget: int, keep_first: int = 0, keep_last: int = 0,
                 status: torch.Tensor | None = None, stream=None):
    """Which tokens of a sequence longer than `budget` stay: the first keep_first, the last
    keep_last, and those of the largest weights [n_seqs, width] among the others.

    Returns (path [n_seqs, budget], n_draft [n_seqs], n_keep [n_seqs], weights): the
    first three make ibp_kv_accept(pool, table, lens, refs, n_draft, path, n_keep) move
    what stays to the front; the weights have moved already.  The move rewrites the
    sequence's pages: one that shares them with a fork is left alone by it (status
    IBP_EINVAL), one longer than its weights by this call (status IBP_ERANGE)."""
    lib = _load()

    def check():
        _on_device("lens", lens)
        _ints("lens", lens, None)
        _floats("weights", weights, lens.shape[0], None)
        return weights.shape

    if not 1 <= budget < 1 << 31 or keep_first < 0 or keep_last < 0 or keep_first + keep_last > budget:
        raise ValueError("budget must be 1 or more and hold keep_first >= 0 and keep_last >= 0 tokens")
    device = weights.device
    handle, where = _for(stream, device)
    with where:
        n, width = _once(("evict", _form(weights), _form(lens)), check)
        path = torch.empty((n, budget), dtype=torch.int32, device=device)
        n_draft, n_keep = (torch.empty(n, dtype=torch.int32, device=device) for _ in range(2))
        out = torch.empty_like(weights)
        _check(lib.ibp_kv_evict(weights.data_ptr(), width, lens.data_ptr(), n, budget, keep_first, keep_last,
                                path.data_ptr(), n_draft.data_ptr(), n_keep.data_ptr(), out.data_ptr(),
                                _status(status, device), handle), "ibp_kv_evict")
    return path, n_draft, n_keep, _result("ibp_kv_evict", out, weights)
