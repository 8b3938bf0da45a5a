"""The paged key/value cache: planning a step, appending to it, attention over it.

A serving program whose products run on compressed weights
(``decode_gemm``) holds its keys and values in pages of a cache.  Per step,
``paged_plan`` finds the pages and slots of the new tokens from the requests'
lengths; per layer, ``paged_append`` rotates, rounds and stores the step's
keys and values and ``paged_attention`` attends over everything stored.
Lengths, tables and cursors stay on the device; nothing waits for the GPU.

Like the rest of the package this module only checks and marshals arguments
for the C ABI (``include/dfc.h``).
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple

import torch

from . import _check, library

__all__ = ["PagedPlan", "paged_plan", "paged_append", "paged_attention", "paged_attention_workspace"]

_DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

# The argument structures of include/dfc.h, packed in one go: filling a ctypes
# structure field by field takes longer than the smaller kernels run.
_CACHE = "QQ6q5I4x"
CACHE = struct.Struct("=" + _CACHE)
PLAN_ARGS = struct.Struct("=4I4Qq8Q")
APPEND_ARGS = struct.Struct("=" + _CACHE + "QQQ4qQIIQQ4qIII4xQQQ")
ATTENTION_ARGS = struct.Struct("=" + _CACHE + "4IQQQ4qQQqQQfII4xQQQ")


class PagedPlan(NamedTuple):
    """What ``paged_plan`` gives: device tensors."""
    seq_lens: torch.Tensor   # int32 (requests): tokens held after the step
    cu_q: torch.Tensor       # int32 (requests + 1): prefix sums of the new tokens
    slots: torch.Tensor      # int64 (tokens): cache slot, -1 = none
    positions: torch.Tensor  # int32 (tokens): position in the request
    cursor: torch.Tensor     # int64 (2): the ring's cursor after the step


_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        lib = library()
        for name in ("dfc_paged_plan", "dfc_paged_append", "dfc_paged_attention"):
            fn = getattr(lib, name)
            fn.argtypes = [ctypes.c_char_p, ctypes.c_void_p]
            fn.restype = ctypes.c_int
        lib.dfc_paged_attention_workspace.argtypes = [ctypes.c_char_p, ctypes.POINTER(ctypes.c_uint64)]
        lib.dfc_paged_attention_workspace.restype = ctypes.c_int
        _LIB = lib
    return _LIB


def _device(t, name):
    """The device of the call's main tensor, which must be the current one:
    the launch goes to it."""
    dev = t.get_device()
    if dev < 0:
        raise TypeError(f"{name} must be a device (cuda) tensor")
    if dev != torch.cuda.current_device():
        raise ValueError(f"{name} is on device {dev}, not the current one")
    return dev


def _stream_of(stream, dev):
    if stream is not None:
        return int(stream)
    return torch._C._cuda_getCurrentRawStream(dev)


def _vector(t, dtype, n, dev, name):
    """Device address of a contiguous vector of n elements."""
    if t.dtype is not dtype or t.dim() != 1 or t.get_device() != dev or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous one-dimensional {dtype} tensor on the call's device")
    if t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} elements, not {n}")
    return t.data_ptr()


def _rows(t, name, dtype, shape, dev):
    """Device address and strides of (tokens, heads, head_dim) rows: any
    strides of the first two dimensions, the last one contiguous."""
    if t.dtype is not dtype or t.get_device() != dev or t.dim() != 3:
        raise TypeError(f"{name} must be a {dtype} tensor of shape (tokens, heads, head_dim) on the call's device")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    s0, s1, s2 = t.stride()
    if s2 != 1 and shape[2] != 1:
        raise ValueError(f"the values of a head of {name} must be contiguous")
    return t.data_ptr(), s0, s1


def _cache(k, v, dev):
    """The fields of dfc_paged_cache."""
    dtype, shape = k.dtype, k.shape
    if len(shape) != 4 or shape != v.shape or dtype is not v.dtype or k.get_device() != dev or v.get_device() != dev:
        raise TypeError("k_cache and v_cache must be tensors of one shape (pages, page size, heads, head_dim) and one "
                        "type on the call's device")
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError("the cache must be bfloat16 or float16")
    k0, k1, k2, k3 = k.stride()
    v0, v1, v2, v3 = v.stride()
    if k3 != 1 or v3 != 1:
        raise ValueError("the values of a head must be contiguous in the cache")
    return (k.data_ptr(), v.data_ptr(), k0, k1, k2, v0, v1, v2, *shape, _DTYPE[dtype])


def _table(t, n, dev):
    """Device address, row stride and width of a block table of n rows."""
    if t.dim() != 2 or t.dtype is not torch.int32 or t.get_device() != dev:
        raise TypeError("block_table must be an int32 tensor of shape (requests, pages) on the call's device")
    rows, width = t.shape
    s0, s1 = t.stride()
    if rows != n:
        raise ValueError(f"block_table has {rows} rows for {n} requests")
    if s1 != 1 and width > 1:
        raise ValueError("the entries of a row of block_table must be contiguous")
    # a single row's stride says nothing
    return t.data_ptr(), s0 if n > 1 else width, width


def _status(t, dev):
    if t is None:
        return 0
    if t.get_device() != dev or t.element_size() != 4 or t.numel() < 1:
        raise ValueError("status must be a device tensor of at least one 32-bit element")
    return t.data_ptr()


def _count(x, name):
    """A size that the C structures hold in 32 bits."""
    if not 0 <= x < 1 << 31:
        raise ValueError(f"{name} must be between 0 and 2^31 - 1")
    return x


def _keep(stream, dev, *tensors):
    """Tensors allocated here are used on the caller's stream."""
    if stream is not None:
        ext = torch.cuda.ExternalStream(int(stream), device=dev)
        for t in tensors:
            t.record_stream(ext)


def paged_plan(context_lens, new_lens, block_table, free_pages, cursor, page_size: int, tokens: int, out=None,
               status=None, stream=None) -> PagedPlan:
    """Pages, slots and positions of a step, from its request lengths.

    ``context_lens`` / ``new_lens``: int32 device vectors, tokens every request
    holds and brings.  ``block_table``: int32 (requests, max pages); a request
    of c tokens holds its first ceil(c / page_size) entries, and the pages it
    needs beyond them are taken off the ring and written behind them.
    ``free_pages``: int32 ring of page numbers, ``cursor``: int64 {head, tail}
    (free are entries head .. tail - 1 modulo the ring's length).  ``tokens``:
    the length of the slots and positions, at least the step's new tokens (the
    rest become -1 and 0).  ``out``: a ``PagedPlan`` to write into (a captured
    step's buffers; its cursor may not be ``cursor``).  Asynchronous."""
    dev = _device(block_table, "block_table")
    n = context_lens.shape[0] if context_lens.dim() == 1 else -1
    table, table_stride, width = _table(block_table, n, dev)
    _count(page_size, "page_size")
    _count(tokens, "tokens")
    i32, i64 = torch.int32, torch.int64
    inputs = (_vector(context_lens, i32, n, dev, "context_lens"), _vector(new_lens, i32, n, dev, "new_lens"), table,
              table_stride, _vector(free_pages, i32, free_pages.shape[0], dev, "free_pages"),
              _vector(cursor, i64, 2, dev, "cursor"))
    if out is None:
        # two allocations rather than five
        narrow = torch.empty(2 * n + 1 + tokens, dtype=i32, device=dev)
        wide = torch.empty(tokens + 2, dtype=i64, device=dev)
        _keep(stream, dev, narrow, wide)
        at = narrow.data_ptr()
        seq_lens, cu_q, positions = at, at + 4 * n, at + 4 * (2 * n + 1)
        slots = wide.data_ptr()
        cursor_out = slots + 8 * tokens
        lens, starts, places = narrow.split_with_sizes((n, n + 1, tokens))
        slot_view, cursor_view = wide.split_with_sizes((tokens, 2))
        out = PagedPlan(lens, starts, slot_view, places, cursor_view)
    else:
        seq_lens = _vector(out.seq_lens, i32, n, dev, "the plan's seq_lens")
        cu_q = _vector(out.cu_q, i32, n + 1, dev, "the plan's cu_q")
        slots = _vector(out.slots, i64, tokens, dev, "the plan's slots")
        positions = _vector(out.positions, i32, tokens, dev, "the plan's positions")
        cursor_out = _vector(out.cursor, i64, 2, dev, "the plan's cursor")
    args = PLAN_ARGS.pack(n, width, page_size, free_pages.shape[0], tokens, *inputs, seq_lens, cu_q, slots, positions,
                          cursor_out, _status(status, dev))
    _check(_lib().dfc_paged_plan(args, _stream_of(stream, dev)), "dfc_paged_plan")
    return out


def paged_append(k, v, k_cache, v_cache, slots, q=None, q_out=None, positions=None, rotary=None,
                 interleaved: bool = False, status=None, stream=None):
    """Store a step's keys and values (``k``, ``v``: (tokens, kv_heads,
    head_dim), float32 or the cache's type) in the cache (``k_cache``,
    ``v_cache``: (pages, page size, kv_heads, head_dim), bfloat16 or float16)
    at ``slots`` (int64, -1 = not stored).  With ``rotary`` (float32
    (positions, rot_dim): rot_dim / 2 cosines and as many sines) k is rotated
    by its token's ``positions`` (int32) first, and so is ``q`` (tokens,
    heads, head_dim); the rotated q, in the cache's type, is returned
    (``q_out``, or a new tensor).  Asynchronous."""
    dev = _device(k_cache, "k_cache")
    cache = _cache(k_cache, v_cache, dev)
    tokens, source = k.shape[0], k.dtype
    if source is not torch.float32 and source is not k_cache.dtype:
        raise TypeError("k and v must be float32 or of the cache's type")
    shape = (tokens, cache[10], cache[11])
    k_ptr, k0, k1 = _rows(k, "k", source, shape, dev)
    v_ptr, v0, v1 = _rows(v, "v", source, shape, dev)
    q_heads = q_ptr = q0 = q1 = out_ptr = o0 = o1 = 0
    if q is not None:
        if q.dim() != 3 or q.shape[0] != tokens or q.shape[2] != cache[11]:
            raise ValueError("q must have k's tokens and head_dim")
        q_heads = q.shape[1]
        q_ptr, q0, q1 = _rows(q, "q", source, q.shape, dev)
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=k_cache.dtype, device=dev)
            _keep(stream, dev, q_out)
        out_ptr, o0, o1 = _rows(q_out, "q_out", k_cache.dtype, q.shape, dev)
    rot = angles = max_pos = pos = 0
    if rotary is not None:
        if rotary.dtype is not torch.float32 or rotary.dim() != 2 or rotary.get_device() != dev or \
                not rotary.is_contiguous():
            raise TypeError("rotary must be a contiguous float32 tensor of shape (positions, rot_dim) on the call's "
                            "device")
        if positions is None:
            raise ValueError("rotary needs positions")
        max_pos, rot = rotary.shape
        pos = _vector(positions, torch.int32, tokens, dev, "positions")
        angles = rotary.data_ptr()
    args = APPEND_ARGS.pack(*cache, tokens, k_ptr, v_ptr, k0, k1, v0, v1, _vector(slots, torch.int64, tokens, dev, "slots"),
                            _DTYPE[source], q_heads, q_ptr, out_ptr, q0, q1, o0, o1, rot, 1 if interleaved else 0,
                            max_pos, pos, angles, _status(status, dev))
    _check(_lib().dfc_paged_append(args, _stream_of(stream, dev)), "dfc_paged_append")
    return q_out


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(*sizes):
    """dfc_paged_attention_workspace, a function of sizes alone."""
    page_size, kv_heads, dim, dtype, heads, n, width, max_q_len, tokens = sizes
    args = ATTENTION_ARGS.pack(16, 16, 0, 0, 0, 0, 0, 0, 1, page_size, kv_heads, dim, dtype, heads, n, width, max_q_len,
                               tokens, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 1.0, 0, 0, 0, 0, 0)
    need = ctypes.c_uint64()
    _check(_lib().dfc_paged_attention_workspace(args, ctypes.byref(need)), "dfc_paged_attention_workspace")
    return need.value


def paged_attention_workspace(q, k_cache, v_cache, block_table, cu_q, seq_lens, max_q_len: int = 0) -> int:
    """Device bytes of the workspace ``paged_attention`` uses for these
    arguments (from their shapes alone)."""
    _, page_size, kv_heads, dim = k_cache.shape
    return _workspace_bytes(page_size, kv_heads, dim, _DTYPE[k_cache.dtype], q.shape[1], seq_lens.shape[0],
                            block_table.shape[1], _count(max_q_len, "max_q_len"), q.shape[0])


def paged_attention(q, k_cache, v_cache, block_table, cu_q, seq_lens, scale: float | None = None, causal: bool = True,
                    window: int = 0, max_q_len: int = 0, out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of a step's new tokens (``q``: (tokens, heads, head_dim) in
    the cache's type; request r's are rows cu_q[r] .. cu_q[r + 1] - 1) over
    the first seq_lens[r] tokens of each request in the paged cache, its new
    ones included.  ``scale``: of the scores (None: head_dim ** -0.5).
    ``causal``: a token sees itself and what is before it.  ``window``: it
    sees that many at most (0: all).  ``max_q_len``: the most new tokens of a
    request, if the caller knows (0: unknown; it decides the kernel's shape,
    never its result).  ``lse``: a float32 (tokens, heads) tensor for the log
    of every row's sum of exponentials, or True for a new one.  ``workspace``:
    a device uint8 tensor of at least ``paged_attention_workspace`` bytes that
    nothing else uses until the call's work has run (None: allocated here).
    Returns out, or (out, lse).  Asynchronous."""
    dev = _device(q, "q")
    cache = _cache(k_cache, v_cache, dev)
    dtype = q.dtype
    if dtype is not k_cache.dtype or q.dim() != 3:
        raise TypeError("q must be a tensor of shape (tokens, heads, head_dim) of the cache's type")
    n = seq_lens.shape[0]
    shape = q.shape
    tokens, heads, dim = shape
    if dim != cache[11] or not heads or not cache[10] or heads % cache[10]:
        raise ValueError("q must have the cache's head_dim and a multiple of its heads")
    table, table_stride, width = _table(block_table, n, dev)
    _count(window, "window")
    _count(max_q_len, "max_q_len")
    q_ptr, q0, q1 = _rows(q, "q", dtype, shape, dev)
    if out is None:
        out = torch.empty_like(q) if q.is_contiguous() else torch.empty(shape, dtype=dtype, device=dev)
        _keep(stream, dev, out)
    out_ptr, o0, o1 = _rows(out, "out", dtype, shape, dev)
    lse_ptr = 0
    if lse is True:
        lse = torch.empty((tokens, heads), dtype=torch.float32, device=dev)
        _keep(stream, dev, lse)
        lse_ptr = lse.data_ptr()
    elif lse is not None:
        if lse.dtype is not torch.float32 or lse.shape != shape[:2] or lse.get_device() != dev or \
                not lse.is_contiguous():
            raise TypeError("lse must be a contiguous float32 tensor of shape (tokens, heads) on the call's device")
        lse_ptr = lse.data_ptr()
    if workspace is None:
        workspace = torch.empty(_workspace_bytes(*cache[9:], heads, n, width, max_q_len, tokens), dtype=torch.uint8,
                                device=dev)
        _keep(stream, dev, workspace)
    elif workspace.get_device() != dev or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous tensor on the call's device")
    args = ATTENTION_ARGS.pack(*cache, heads, n, width, max_q_len, tokens, q_ptr, out_ptr, q0, q1, o0, o1, lse_ptr,
                               table, table_stride, _vector(cu_q, torch.int32, n + 1, dev, "cu_q"),
                               _vector(seq_lens, torch.int32, n, dev, "seq_lens"),
                               dim ** -0.5 if scale is None else scale, 1 if causal else 0, window,
                               workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                               _status(status, dev))
    _check(_lib().dfc_paged_attention(args, _stream_of(stream, dev)), "dfc_paged_attention")
    return out if lse is None else (out, lse)
