"""The paged key/value cache: planning a step, appending to it, attention over
it, giving pages back, sharing and moving them; and the next tokens of a step.

A serving program whose products run on compressed weights
(``decode_gemm``) holds its keys and values in pages of a cache.  Per step,
``paged_plan`` finds the pages and slots of the new tokens from the requests'
lengths; per layer, ``paged_append`` norms, rotates, rounds and stores the
step's keys and values and ``paged_attention`` attends over everything stored.
``verify_drafts`` draws the next tokens from the step's logits and says which
drafted ones hold; ``paged_release`` gives the others' pages back, and those of
requests that end and of what a window has passed.  ``paged_fork`` makes
requests copies of others that share their full pages, ``paged_compact`` makes
the held pages dense, ``paged_copy`` copies the pages that either asks for.
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

__all__ = ["PagedPlan", "paged_plan", "paged_append", "paged_attention", "paged_attention_workspace", "PagedFork",
           "PagedMoves", "paged_release", "paged_fork", "paged_compact", "paged_copy", "Verified", "verify_drafts",
           "verify_drafts_workspace"]


class PagedPlan(NamedTuple):
    """What ``paged_plan`` gives: device tensors."""
    seq_lens: torch.Tensor   # int32 (requests): tokens held after the step
    cu_q: torch.Tensor       # int32 (requests + 1): prefix sums of the new tokens
    slots: torch.Tensor      # int64 (tokens): cache slot, -1 = none
    positions: torch.Tensor  # int32 (tokens): position in the request
    cursor: torch.Tensor     # int64 (2): the ring's cursor after the step


class PagedFork(NamedTuple):
    """What ``paged_fork`` gives: device tensors."""
    context_lens: torch.Tensor  # int32 (requests): tokens held after the call
    src: torch.Tensor           # int32 (requests): page to copy for each request, -1 = none
    dst: torch.Tensor           # int32 (requests): where to
    cursor: torch.Tensor        # int64 (2): the ring's cursor after the call


class PagedMoves(NamedTuple):
    """What ``paged_compact`` gives: device tensors."""
    src: torch.Tensor   # int32 (pages / 2): pages to copy, in ascending order, then -1
    dst: torch.Tensor   # int32 (pages / 2): where to
    used: torch.Tensor  # int32 (1): pages held


class Verified(NamedTuple):
    """What ``verify_drafts`` gives: device tensors."""
    accepted: torch.Tensor  # int32 (requests): drafts that hold
    tokens: torch.Tensor    # int64 (requests): the token that follows them, -1 = none


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
                   ("dfc_paged_plan", "dfc_paged_append_normed", "dfc_paged_attention_sinks",
                    "dfc_paged_attention_workspace", "dfc_paged_release", "dfc_paged_fork", "dfc_paged_compact",
                    "dfc_paged_compact_workspace", "dfc_paged_copy", "dfc_verify_drafts", "dfc_verify_workspace")))
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
                 interleaved: bool = False, status=None, stream=None, q_norm=None, k_norm=None, eps: float = 1e-6):
    """Store a step's keys and values (``k``, ``v``: (tokens, kv_heads,
    head_dim), float32 or the cache's type) in the cache (``k_cache``,
    ``v_cache``: (pages, page size, kv_heads, head_dim), bfloat16 or float16)
    at ``slots`` (int64, -1 = not stored).  With ``rotary`` (float32
    (positions, rot_dim): rot_dim / 2 cosines and as many sines) k is rotated
    by its token's ``positions`` (int32) first, and so is ``q`` (tokens,
    heads, head_dim); the rotated q, in the cache's type, is returned
    (``q_out``, or a new tensor).  With ``q_norm`` / ``k_norm`` ((head_dim),
    float32 or the cache's type) every head of q / k is first multiplied by
    them and divided by the root of its mean square plus ``eps``.
    Asynchronous."""
    r = _call(stream, (q_out,), (_BIND or _load()).append, k, v, k_cache, v_cache, slots, q, q_out, positions, rotary,
              interleaved, status, q_norm, k_norm, eps)
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
                    window: int = 0, max_q_len: int = 0, out=None, lse=None, workspace=None, status=None, stream=None,
                    sinks: int = 0):
    """Attention of a step's new tokens (``q``: (tokens, heads, head_dim) in
    the cache's type; request r's are rows cu_q[r] .. cu_q[r + 1] - 1) over
    the first seq_lens[r] tokens of each request in the paged cache, its new
    ones included.  ``scale``: of the scores (None: head_dim ** -0.5).
    ``causal``: a token sees itself and what is before it.  ``window``: it
    sees that many at most (0: all), and with ``sinks`` beside them the first
    so many of its request.  ``max_q_len``: the most new tokens of a
    request, if the caller knows (0: unknown; it decides the kernel's shape
    and so the result within rounding).  ``lse``: a float32 (tokens, heads) tensor for the log
    of every row's sum of exponentials, or True for a new one.  ``workspace``:
    a device uint8 tensor of at least ``paged_attention_workspace`` bytes that
    nothing else uses until the call's work has run (None: allocated here).
    Returns out, or (out, lse).  Asynchronous."""
    r = _call(stream, (out, lse), (_BIND or _load()).attention, q, k_cache, v_cache, block_table, cu_q, seq_lens, scale,
              causal, window, max_q_len, out, lse, workspace, status, sinks)
    if r[0]:
        _check(r[0], "dfc_paged_attention")
    return r[1] if r[2] is None else r[1:]


def paged_release(held_lens, keep_lens, block_table, free_pages, cursor, shared, page_size: int, window: int = 0,
                  sinks: int = 0, out=None, status=None, stream=None):
    """Cut requests to their first ``keep_lens`` of ``held_lens`` tokens (int32
    device vectors; 0 ends a request) and give back the pages that they do not
    need: those behind what is kept and, with a ``window``, those that lie
    wholly between the first ``sinks`` tokens and the window of the next token.
    Their entries in ``block_table`` become -1.  ``free_pages``: the ring that
    ``paged_plan`` takes pages off; pages that nobody holds any more are
    written from its tail on, in ascending order.  ``shared``: int32 (pages of
    the cache), the number of requests beyond the first that hold each page:
    zeros at first, kept by these calls.  Returns the new cursor (``out``, or a
    new int64 tensor; not ``cursor``).  Asynchronous."""
    r = _call(stream, (out,), (_BIND or _load()).release, held_lens, keep_lens, block_table, free_pages, cursor, shared,
              page_size, window, sinks, out, status)
    if r[0]:
        _check(r[0], "dfc_paged_release")
    return r[1] if out is None else out


def paged_fork(context_lens, parents, block_table, free_pages, cursor, shared, page_size: int, fork_lens=None, out=None,
               status=None, stream=None) -> PagedFork:
    """Make requests that hold nothing copies of others: request r gets the
    first ``fork_lens[r]`` tokens (None: all) of request ``parents[r]`` (int32;
    -1: it stays as it is).  Full pages are shared; one that ends inside gets a
    new page off the ring, and the result's ``src`` and ``dst`` say what
    ``paged_copy`` has to copy before the next append.  ``context_lens``,
    ``block_table``, ``free_pages``, ``cursor``, ``shared``: as in
    ``paged_plan`` and ``paged_release``.  ``out``: a ``PagedFork`` to write into
    (its lengths and cursor may not be the inputs).  Asynchronous."""
    r = _call(stream, out or (), (_BIND or _load()).fork, context_lens, parents, block_table, free_pages, cursor, shared,
              page_size, fork_lens, out, status)
    if r[0]:
        _check(r[0], "dfc_paged_fork")
    return PagedFork(*r[1:]) if out is None else out


def paged_compact(context_lens, block_table, free_pages, cursor, shared, page_size: int, out=None, status=None,
                  stream=None) -> PagedMoves:
    """Make the held pages dense: of the pages that requests hold and those on
    the ring together, the held ones come to be the lowest.  Tables, ``shared``
    and the ring (then in ascending order; its cursor stays) are rewritten; the
    result's ``src`` and ``dst`` say what ``paged_copy`` has to copy before the
    next step.  Where ring and tables contradict each other nothing moves.
    ``out``: a ``PagedMoves`` to write into.  Asynchronous."""
    r = _call(stream, out or (), (_BIND or _load()).compact, context_lens, block_table, free_pages, cursor, shared,
              page_size, out, status)
    if r[0]:
        _check(r[0], "dfc_paged_compact")
    return PagedMoves(*r[1:]) if out is None else out


def paged_copy(caches, src, dst, status=None, stream=None) -> None:
    """Copy the keys and values of page ``src[i]`` to page ``dst[i]`` (int32
    device vectors; negative: none) in every one of ``caches``, a sequence of
    pairs (k_cache, v_cache) of one shape, layout and type: the layers of a
    model.  Destinations are distinct and no sources.  Asynchronous."""
    r = _call(stream, (), (_BIND or _load()).copy, caches, src, dst, status)
    _check(r[0], "dfc_paged_copy")


def verify_drafts_workspace(logits, cu_rows, draft_logits=None) -> int:
    """Device bytes of the workspace ``verify_drafts`` uses for these arguments
    (from their shapes alone)."""
    status, size = (_BIND or _load()).verify_workspace(logits, cu_rows, draft_logits)
    _check(status, "dfc_verify_workspace")
    return size


def verify_drafts(logits, cu_rows, drafts, uniforms, draft_logits=None, temperature=None, out=None, workspace=None,
                  status=None, stream=None) -> Verified:
    """Which drafted tokens hold, and the token that follows them.  Request r's
    rows of ``logits`` ((rows, vocabulary), float32, bfloat16 or float16) are
    cu_rows[r] .. cu_rows[r + 1] - 1 (int32), one more than it has drafts:
    ``drafts[i]`` (int64) is the token drafted to follow row i, and the last
    row's entry is not read.  ``draft_logits``: what the drafts were drawn from,
    row by row (None: they are certain, as of a lookup).  ``temperature``:
    float32 (requests), of both logits; None: 1; 0: the largest logit.
    ``uniforms``: float32 (rows) in [0, 1); a request's last one draws its
    token, the others try its drafts, so that every answer is distributed as
    if drawn from ``logits`` token by token.  A request with one row: a token
    drawn from it.  ``workspace``: a device tensor of at least
    ``verify_drafts_workspace`` bytes that nothing else uses until the call's
    work has run (None: allocated here).  ``out``: a ``Verified`` to write into.
    Asynchronous."""
    r = _call(stream, out or (), (_BIND or _load()).verify, logits, cu_rows, drafts, uniforms, draft_logits, temperature,
              out, workspace, status)
    if r[0]:
        _check(r[0], "dfc_verify_drafts")
    return Verified(*r[1:]) if out is None else out
