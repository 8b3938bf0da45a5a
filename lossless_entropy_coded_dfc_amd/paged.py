"""The paged key/value cache: planning a step, appending to it, attention over it.

A serving program whose products run on compressed weights
(``decode_gemm``) holds its keys and values in pages of a cache.  Per step,
``paged_plan`` finds the pages and slots of the new tokens from the requests'
lengths; per layer, ``paged_append`` rotates, rounds and stores the step's
keys and values and ``paged_attention`` attends over everything stored.
Lengths, tables and cursors stay on the device; nothing waits for the GPU.
There is no backward pass: tensors that require a gradient are refused, unless
gradients are off (``torch.no_grad()``).  ``stream``: the handle of the stream
that a call's work goes to (None: torch's current one); what the call allocates
is that stream's memory.

The checks of the arguments and their marshalling for the C ABI
(``include/dfc.h``) are ``csrc/dfc_paged_bind.cpp``: done in Python, they take
longer than the smaller kernels run.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

from . import DfcLibraryMissing, _allocating_for, _check, library

__all__ = ["PagedPlan", "paged_plan", "paged_append", "paged_attention", "paged_attention_workspace"]


class PagedPlan(NamedTuple):
    """What ``paged_plan`` gives: device tensors."""
    seq_lens: torch.Tensor   # int32 (requests): tokens held after the step
    cu_q: torch.Tensor       # int32 (requests + 1): prefix sums of the new tokens
    slots: torch.Tensor      # int64 (tokens): cache slot, -1 = none
    positions: torch.Tensor  # int32 (tokens): position in the request
    cursor: torch.Tensor     # int64 (2): the ring's cursor after the step


_BIND = None


def _load():
    """The binding, told where libdfc.so's functions are."""
    global _BIND
    try:
        from . import _paged
    except ImportError as e:
        raise DfcLibraryMissing(f"{os.path.join(os.path.dirname(__file__), '_paged.so')} cannot be loaded ({e}); run "
                                "`python -c 'import __graft_entry__ as g; g.build()'`") from e
    built = getattr(_paged, "torch_version", "of another build")
    if built != torch.__version__:
        raise DfcLibraryMissing(f"_paged.so is built against torch {built}, not {torch.__version__}; build it again")
    lib = library()
    _paged.setup(torch._C._cuda_getCurrentRawStream,
                 *(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in
                   ("dfc_paged_plan", "dfc_paged_append", "dfc_paged_attention", "dfc_paged_attention_workspace")))
    _BIND = _paged
    return _paged


def _call(stream, given, entry, *args):
    """An entry of the binding, which allocates the workspace and the results
    that are not ``given``, with its work on ``stream``.  What was allocated
    for another stream than the current one counts as used on the current one
    too, where the caller goes on with it: its memory is not handed to the
    other stream's later work while the current one may still read it."""
    if stream is None:
        return entry(*args, None)
    current = torch.cuda.current_stream()
    with _allocating_for(stream):
        r = entry(*args, stream)
    for t in r[1:]:
        if t is not None and not any(t is g for g in given):
            t.record_stream(current)
    return r


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
    r = _call(stream, out or (), (_BIND or _load()).plan, context_lens, new_lens, block_table, free_pages, cursor,
              page_size, tokens, out, status)
    if r[0]:
        _check(r[0], "dfc_paged_plan")
    return PagedPlan(*r[1:]) if out is None else out


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
    r = _call(stream, (q_out,), (_BIND or _load()).append, k, v, k_cache, v_cache, slots, q, q_out, positions, rotary,
              interleaved, status)
    if r[0]:
        _check(r[0], "dfc_paged_append")
    return r[1]


def paged_attention_workspace(q, k_cache, v_cache, block_table, cu_q, seq_lens, max_q_len: int = 0) -> int:
    """Device bytes of the workspace ``paged_attention`` uses for these
    arguments (from their shapes alone)."""
    status, size = (_BIND or _load()).workspace(q, k_cache, v_cache, block_table, seq_lens, max_q_len)
    _check(status, "dfc_paged_attention_workspace")
    return size


def paged_attention(q, k_cache, v_cache, block_table, cu_q, seq_lens, scale: float | None = None, causal: bool = True,
                    window: int = 0, max_q_len: int = 0, out=None, lse=None, workspace=None, status=None, stream=None):
    """Attention of a step's new tokens (``q``: (tokens, heads, head_dim) in
    the cache's type; request r's are rows cu_q[r] .. cu_q[r + 1] - 1) over
    the first seq_lens[r] tokens of each request in the paged cache, its new
    ones included.  ``scale``: of the scores (None: head_dim ** -0.5).
    ``causal``: a token sees itself and what is before it.  ``window``: it
    sees that many at most (0: all).  ``max_q_len``: the most new tokens of a
    request, if the caller knows (0: unknown; it decides the kernel's shape
    and so the result within rounding).  ``lse``: a float32 (tokens, heads) tensor for the log
    of every row's sum of exponentials, or True for a new one.  ``workspace``:
    a device uint8 tensor of at least ``paged_attention_workspace`` bytes that
    nothing else uses until the call's work has run (None: allocated here).
    Returns out, or (out, lse).  Asynchronous."""
    r = _call(stream, (out, lse), (_BIND or _load()).attention, q, k_cache, v_cache, block_table, cu_q, seq_lens, scale,
              causal, window, max_q_len, out, lse, workspace, status)
    if r[0]:
        _check(r[0], "dfc_paged_attention")
    return r[1] if r[2] is None else r[1:]
