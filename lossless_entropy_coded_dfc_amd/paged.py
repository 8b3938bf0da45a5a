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
from typing import NamedTuple

import torch

from . import _check, _status_ptr, _stream, library

__all__ = ["PagedPlan", "paged_plan", "paged_append", "paged_attention", "paged_attention_workspace"]

BF16, F16, F32 = 0, 1, 2
_DTYPE = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}

_i64x2, _i64x3 = ctypes.c_int64 * 2, ctypes.c_int64 * 3
_ptr, _u32, _u64, _i64 = ctypes.c_void_p, ctypes.c_uint32, ctypes.c_uint64, ctypes.c_int64


class Cache(ctypes.Structure):
    _fields_ = [("k_dev", _ptr), ("v_dev", _ptr), ("k_stride", _i64x3), ("v_stride", _i64x3), ("n_pages", _u32),
                ("page_size", _u32), ("kv_heads", _u32), ("head_dim", _u32), ("dtype", _u32)]


class PlanArgs(ctypes.Structure):
    _fields_ = [("n_requests", _u32), ("max_pages", _u32), ("page_size", _u32), ("n_ring", _u32), ("tokens", _u64),
                ("context_lens", _ptr), ("new_lens", _ptr), ("block_table", _ptr), ("table_stride", _i64),
                ("free_pages", _ptr), ("cursor", _ptr), ("seq_lens", _ptr), ("cu_q", _ptr), ("slots", _ptr),
                ("positions", _ptr), ("cursor_out", _ptr), ("status_dev", _ptr)]


class AppendArgs(ctypes.Structure):
    _fields_ = [("cache", Cache), ("tokens", _u64), ("k_dev", _ptr), ("v_dev", _ptr), ("k_src_stride", _i64x2),
                ("v_src_stride", _i64x2), ("slots", _ptr), ("source_dtype", _u32), ("q_heads", _u32), ("q_dev", _ptr),
                ("q_out_dev", _ptr), ("q_stride", _i64x2), ("q_out_stride", _i64x2), ("rot_dim", _u32),
                ("interleaved", _u32), ("max_positions", _u32), ("positions", _ptr), ("rotary_dev", _ptr),
                ("status_dev", _ptr)]


class AttentionArgs(ctypes.Structure):
    _fields_ = [("cache", Cache), ("heads", _u32), ("n_requests", _u32), ("max_pages", _u32), ("max_q_len", _u32),
                ("tokens", _u64), ("q_dev", _ptr), ("out_dev", _ptr), ("q_stride", _i64x2), ("out_stride", _i64x2),
                ("lse_dev", _ptr), ("block_table", _ptr), ("table_stride", _i64), ("cu_q", _ptr), ("seq_lens", _ptr),
                ("scale", ctypes.c_float), ("causal", _u32), ("window", _u32), ("workspace_dev", _ptr),
                ("workspace_bytes", _u64), ("status_dev", _ptr)]


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
        for name, args in (("dfc_paged_plan", PlanArgs), ("dfc_paged_append", AppendArgs),
                           ("dfc_paged_attention", AttentionArgs)):
            fn = getattr(lib, name)
            fn.argtypes = [ctypes.POINTER(args), _ptr]
            fn.restype = ctypes.c_int
        lib.dfc_paged_attention_workspace.argtypes = [ctypes.POINTER(AttentionArgs), ctypes.POINTER(_u64)]
        lib.dfc_paged_attention_workspace.restype = ctypes.c_int
        _LIB = lib
    return _LIB


def _vector(t, dtype, n, name):
    """Device address of a contiguous vector of n elements (None: any number)."""
    if t.dtype != dtype or t.dim() != 1 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous one-dimensional {dtype} device tensor")
    if n is not None and t.shape[0] != n:
        raise ValueError(f"{name} has {t.shape[0]} elements, not {n}")
    return t.data_ptr()


def _rows(t, name, dtype, shape=None):
    """Device address of (tokens, heads, head_dim) rows: any strides of the
    first two dimensions, the last one contiguous."""
    if t.dim() != 3 or not t.is_cuda or t.dtype != dtype:
        raise TypeError(f"{name} must be a {dtype} device tensor of shape (tokens, heads, head_dim)")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, not {shape}")
    if t.stride(2) != 1 and t.shape[2] != 1:
        raise ValueError(f"the values of a head of {name} must be contiguous")
    return t.data_ptr()


def _cache(k, v):
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.device != v.device or not k.is_cuda:
        raise TypeError("k_cache and v_cache must be device tensors of one shape (pages, page size, heads, head_dim), "
                        "one type and one device")
    if k.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("the cache must be bfloat16 or float16")
    if k.stride(3) != 1 or v.stride(3) != 1:
        raise ValueError("the values of a head must be contiguous in the cache")
    pages, size, heads, dim = k.shape
    return Cache(k.data_ptr(), v.data_ptr(), _i64x3(*k.stride()[:3]), _i64x3(*v.stride()[:3]), pages, size, heads, dim,
                 _DTYPE[k.dtype])


def _table(block_table, n_requests):
    if block_table.dim() != 2 or block_table.dtype != torch.int32 or not block_table.is_cuda:
        raise TypeError("block_table must be an int32 device tensor of shape (requests, pages)")
    if block_table.shape[0] != n_requests:
        raise ValueError(f"block_table has {block_table.shape[0]} rows for {n_requests} requests")
    if block_table.shape[1] > 1 and block_table.stride(1) != 1:
        raise ValueError("the entries of a row of block_table must be contiguous")
    # a single row's stride says nothing
    return max(block_table.stride(0), block_table.shape[1]) if n_requests <= 1 else block_table.stride(0)


def _keep(tensor, stream):
    """A tensor allocated here is used on the caller's stream."""
    if stream is not None:
        tensor.record_stream(torch.cuda.ExternalStream(int(stream), device=tensor.device))


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
    n = context_lens.shape[0] if context_lens.dim() == 1 else -1
    table_stride = _table(block_table, n)
    dev = block_table.device
    if out is None:
        whole = torch.empty(2 * n + 1 + tokens, dtype=torch.int32, device=dev)
        wide = torch.empty(tokens + 2, dtype=torch.int64, device=dev)
        out = PagedPlan(whole[:n], whole[n: 2 * n + 1], wide[:tokens], whole[2 * n + 1:], wide[tokens:])
        _keep(whole, stream)
        _keep(wide, stream)
    args = PlanArgs(n, block_table.shape[1], page_size, free_pages.shape[0], tokens,
                    _vector(context_lens, torch.int32, n, "context_lens"), _vector(new_lens, torch.int32, n, "new_lens"),
                    block_table.data_ptr(), table_stride, _vector(free_pages, torch.int32, None, "free_pages"),
                    _vector(cursor, torch.int64, 2, "cursor"), _vector(out.seq_lens, torch.int32, n, "seq_lens"),
                    _vector(out.cu_q, torch.int32, n + 1, "cu_q"), _vector(out.slots, torch.int64, tokens, "slots"),
                    _vector(out.positions, torch.int32, tokens, "positions"),
                    _vector(out.cursor, torch.int64, 2, "the plan's cursor"), _status_ptr(status))
    _check(_lib().dfc_paged_plan(ctypes.byref(args), _stream(stream)), "dfc_paged_plan")
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
    cache = _cache(k_cache, v_cache)
    tokens = k.shape[0]
    shape = (tokens, cache.kv_heads, cache.head_dim)
    source = k.dtype
    if source != torch.float32 and source != k_cache.dtype:
        raise TypeError("k and v must be float32 or of the cache's type")
    args = AppendArgs(cache, tokens, _rows(k, "k", source, shape), _rows(v, "v", source, shape),
                      _i64x2(*k.stride()[:2]), _i64x2(*v.stride()[:2]), _vector(slots, torch.int64, tokens, "slots"),
                      _DTYPE[source], 0)
    if q is not None:
        args.q_dev = _rows(q, "q", source)
        if q.shape[0] != tokens or q.shape[2] != cache.head_dim:
            raise ValueError("q must have k's tokens and head_dim")
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=k_cache.dtype, device=q.device)
            _keep(q_out, stream)
        args.q_heads = q.shape[1]
        args.q_out_dev = _rows(q_out, "q_out", k_cache.dtype, tuple(q.shape))
        args.q_stride = _i64x2(*q.stride()[:2])
        args.q_out_stride = _i64x2(*q_out.stride()[:2])
    if rotary is not None:
        if rotary.dtype != torch.float32 or rotary.dim() != 2 or not rotary.is_cuda or not rotary.is_contiguous():
            raise TypeError("rotary must be a contiguous float32 device tensor of shape (positions, rot_dim)")
        if positions is None:
            raise ValueError("rotary needs positions")
        args.rot_dim = rotary.shape[1]
        args.interleaved = 1 if interleaved else 0
        args.max_positions = rotary.shape[0]
        args.positions = _vector(positions, torch.int32, tokens, "positions")
        args.rotary_dev = rotary.data_ptr()
    args.status_dev = _status_ptr(status)
    _check(_lib().dfc_paged_append(ctypes.byref(args), _stream(stream)), "dfc_paged_append")
    return q_out


def _attention_args(q, k_cache, v_cache, block_table, cu_q, seq_lens, scale, causal, window, max_q_len):
    cache = _cache(k_cache, v_cache)
    n = seq_lens.shape[0]
    q_ptr = _rows(q, "q", k_cache.dtype)
    tokens, heads, dim = q.shape
    if dim != cache.head_dim or heads % cache.kv_heads or not heads:
        raise ValueError("q must have the cache's head_dim and a multiple of its heads")
    if window < 0 or max_q_len < 0:
        raise ValueError("window and max_q_len may not be negative")
    args = AttentionArgs(cache, heads, n, block_table.shape[1], max_q_len, tokens, q_ptr)
    args.q_stride = _i64x2(*q.stride()[:2])
    args.table_stride = _table(block_table, n)
    args.block_table = block_table.data_ptr()
    args.cu_q = _vector(cu_q, torch.int32, n + 1, "cu_q")
    args.seq_lens = _vector(seq_lens, torch.int32, n, "seq_lens")
    args.scale = dim ** -0.5 if scale is None else scale
    args.causal = 1 if causal else 0
    args.window = window
    return args


def paged_attention_workspace(q, k_cache, v_cache, block_table, cu_q, seq_lens, max_q_len: int = 0) -> int:
    """Device bytes of the workspace ``paged_attention`` uses for these
    arguments (from their shapes alone)."""
    args = _attention_args(q, k_cache, v_cache, block_table, cu_q, seq_lens, None, True, 0, max_q_len)
    need = _u64()
    _check(_lib().dfc_paged_attention_workspace(ctypes.byref(args), ctypes.byref(need)),
           "dfc_paged_attention_workspace")
    return need.value


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
    args = _attention_args(q, k_cache, v_cache, block_table, cu_q, seq_lens, scale, causal, window, max_q_len)
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        _keep(out, stream)
    args.out_dev = _rows(out, "out", q.dtype, tuple(q.shape))
    args.out_stride = _i64x2(*out.stride()[:2])
    if lse is True:
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        _keep(lse, stream)
    if lse is not None:
        if lse.dtype != torch.float32 or lse.shape != q.shape[:2] or not lse.is_cuda or not lse.is_contiguous():
            raise TypeError("lse must be a contiguous float32 device tensor of shape (tokens, heads)")
        args.lse_dev = lse.data_ptr()
    if workspace is None:
        need = _u64()
        _check(_lib().dfc_paged_attention_workspace(ctypes.byref(args), ctypes.byref(need)),
               "dfc_paged_attention_workspace")
        workspace = torch.empty(need.value, dtype=torch.uint8, device=q.device)
        _keep(workspace, stream)
    elif not workspace.is_cuda or not workspace.is_contiguous():
        raise TypeError("workspace must be a contiguous device tensor")
    args.workspace_dev = workspace.data_ptr()
    args.workspace_bytes = workspace.numel() * workspace.element_size()
    args.status_dev = _status_ptr(status)
    _check(_lib().dfc_paged_attention(ctypes.byref(args), _stream(stream)), "dfc_paged_attention")
    return out if lse is None else (out, lse)
