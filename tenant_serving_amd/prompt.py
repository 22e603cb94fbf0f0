"""Python binding of the attention of a prompt's tokens (include/bitdelta_step.h): whole prompts, chunks behind what the
cache holds already, a few proposed tokens at a time, over the same paged cache as ``bd_attend``.

Argument marshalling only; there is no fallback.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import step
from .bitdelta import _check, _workspace
from .step import (BD_BF16, _at, _attend_to, _cache, _cap, _given, _index, _overlap, _plain, _refuse_on_cache, _rows,
                   _same_gpu, _Scores, _tensor, bd_kv_cache)


def _refuse_prompt(q, kv, page_table, lengths, starts, slopes, first, last, out, lse, T, heads):
    """The checks of a prompt's tensors, in full; raises or returns."""
    if heads < 1 or heads > 65535 or heads % kv.num_heads:
        raise ValueError("q's heads must be a multiple of the cache's %d, at most 65535 (got %d)"
                         % (kv.num_heads, heads))
    _tensor("page_table", page_table)
    if page_table.dtype != torch.int32:
        raise TypeError("page_table must be torch.int32 (got %s)" % page_table.dtype)
    if page_table.dim() != 2 or page_table.shape[1] < 1:
        raise ValueError("page_table must be [B, max_pages] (got %s)" % (tuple(page_table.shape),))
    if page_table.shape[1] > 1 and page_table.stride(1) != 1:
        raise ValueError("page_table's rows must be contiguous")
    if page_table.shape[1] * kv.page_size > 1 << 24:
        raise ValueError("page_table holds more than 2^24 tokens per sequence")
    B = page_table.shape[0]
    _plain("lengths", lengths, torch.int32, (B,))
    _plain("starts", starts, torch.int32, (B + 1,))
    if T * heads > 1 << 29 or B * kv.num_heads > 1 << 22:
        raise ValueError("at most 2^29 query rows and 2^22 key-value heads of all sequences (got %d, %d)"
                         % (T * heads, B * kv.num_heads))
    if slopes is not None:
        _plain("slopes", slopes, torch.float32, (heads,))
    for name, t in (("first", first), ("last", last)):
        if t is not None:
            _plain(name, t, torch.int32, (T,))
    if out is not None:
        _plain("out", out, torch.bfloat16, (T, heads, kv.head_dim))
    if lse is not None:
        _plain("lse", lse, torch.float32, (T, heads))
    every = (("q", q), ("page_table", page_table), ("lengths", lengths), ("starts", starts), ("slopes", slopes),
             ("first", first), ("last", last), ("out", out), ("lse", lse))
    given = [(name, t) for name, t in every if t is not None and t.numel()]
    for name, t in given:
        for other, o in given:
            if name in ("out", "lse") and other != name and _overlap(t, o):
                raise ValueError("%s overlaps %s" % (name, other))
    _refuse_on_cache(kv, [(name, t) for name, t in given if name in ("out", "lse")])
    _same_gpu(kv.device, every)


def bd_attend_prompt(q: torch.Tensor, kv: bd_kv_cache, page_table: torch.Tensor, lengths: torch.Tensor,
                     starts: torch.Tensor, scale: float | None = None, cap: float | None = None,
                     slopes: torch.Tensor | None = None, first: torch.Tensor | None = None,
                     last: torch.Tensor | None = None, out: torch.Tensor | None = None,
                     lse: torch.Tensor | None = None):
    """softmax(scores) v of several new tokens per sequence over the cache; bf16 [T, num_q_heads, head_dim].

    q [T, num_q_heads, head_dim] is bf16 (any token and head strides) and holds the new tokens of all sequences, one
    after another: those of sequence b are starts[b] .. starts[b + 1] (int32 [B + 1]), and they are the last of its
    lengths[b] tokens (int32 [B]), whose keys and values are in the cache by then, at the pages of page_table
    (int32 [B, max_pages], rows may be strided).  Each sees its sequence up to itself, unless first and last (int32 [T])
    say otherwise: then token t sees the keys first[t] <= j < last[t] of its sequence.  That is a window, a document of
    several in one prompt, or a prefix that sees itself both ways.

    scale defaults to head_dim^-0.5; cap makes cap · tanh(score / cap) of the scores, and slopes (fp32 [num_q_heads])
    takes slopes · distance off them after that.  A token that sees nothing gets zeros; rows of out outside
    starts[0] .. starts[B] are not written (undefined where out is allocated here).  lse, if given, is an fp32
    [T, num_q_heads] tensor that receives the log of the softmax's sum.  out and lse lie apart from each other and from
    all that is read."""
    _cache(kv)
    kind, qs, T, heads, reach = _rows("q", q, None, kv.head_dim)
    if kind != BD_BF16:
        raise TypeError("q must be torch.bfloat16 (got %s)" % q.dtype)
    dev = kv._dev
    scale = kv.head_dim ** -0.5 if scale is None else float(scale)
    if not abs(scale) <= 2.0 ** 60:
        raise ValueError("scale must be at most 2^60 (got %r)" % scale)
    limit, q0 = _cap(cap), q.data_ptr()
    more = [t for t in (starts, slopes, first, last) if t is not None]
    if not (type(page_table) is torch.Tensor and page_table.dim() == 2 and page_table.dtype is torch.int32
            and page_table.is_contiguous() and 1 <= page_table.shape[1] <= (1 << 24) // kv.page_size
            and page_table.get_device() == dev and _index("lengths", lengths, page_table.shape[0], dev)
            and _index("starts", starts, page_table.shape[0] + 1, dev) and q.get_device() == dev
            and 1 <= heads <= 65535 and heads % kv.num_heads == 0
            and T * heads <= 1 << 29 and page_table.shape[0] * kv.num_heads <= 1 << 22
            and (slopes is None or _given(slopes, torch.float32, (heads,), dev))
            and (first is None or _index("first", first, T, dev)) and (last is None or _index("last", last, T, dev))
            and (out is None and lse is None
                 or _attend_to(kv, q0, q0 + reach * 2, page_table, lengths, out, lse, T, heads, dev, more))):
        _refuse_prompt(q, kv, page_table, lengths, starts, slopes, first, last, out, lse, T, heads)
    if step._current_device() != dev:
        with torch.cuda.device(dev):
            return bd_attend_prompt(q, kv, page_table, lengths, starts, scale, cap, slopes, first, last, out, lse)
    lib = step._declared or step._library()
    B, pages = page_table.shape
    nbytes = _prompt_bytes(T, B, heads, kv.num_heads, kv.head_dim, kv.page_size, pages)
    if out is None:
        out = torch.empty((T, heads, kv.head_dim), dtype=torch.bfloat16, device=kv.device)
    ws = _workspace(nbytes, kv.device)
    scores = None
    if cap is not None or more[1:]:
        scores = ctypes.byref(_Scores(limit, _at(slopes), _at(first), _at(last)))
    st = lib.bd_attend_prompt(kv._ref, q0, qs, heads, T, page_table.data_ptr(), page_table.stride(0) if B > 1 else 0,
                              pages, lengths.data_ptr(), starts.data_ptr(), B, scale, scores, out.data_ptr(),
                              lse.data_ptr() if lse is not None else None, ws.data_ptr() if ws is not None else None,
                              nbytes, step._stream_of(dev))
    if st:
        _check(lib, "bd_attend_prompt", st)
    return out


@functools.lru_cache(maxsize=4096)
def _prompt_bytes(*sizes):
    """The library's answer for these sizes: a host function of nothing else."""
    return step._library().bd_attend_prompt_workspace_bytes(*sizes)
