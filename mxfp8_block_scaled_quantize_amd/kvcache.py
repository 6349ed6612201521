"""A paged key-value cache in MXFP4, and the attention over it.

``new`` makes a cache, ``pool`` the stack of its free pages; ``extend`` gives
requests the pages for their new tokens and says in which slot and at which
position each stands, ``release`` takes finished requests' pages back; ``append``
writes keys and values to their slots, ``read`` returns them; ``attention`` answers
queries that stand at the ends of their sequences.  All numbers that change from
step to step (lengths, tables, slots) stay on the device: nothing waits for the
GPU, and a step can be captured in a graph.

The kernels are those of ``include/kvcache.h`` (``kv_*`` mirror it); there is no
fallback.  The cache has no gradient: tensors that require one are refused while
gradients are enabled.  A tensor that a call writes in place (cache, table, free,
out) counts as modified.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, _p, _s
from ._tensors import declare, extension, on_stream

EXPORTED = ("kv_extend", "kv_release", "kv_append", "kv_read", "kv_attention_workspace_bytes", "kv_attention")

_fn = {}


def _functions():
    if not _fn:
        P, I64, I32, F32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
        got = {"kv_extend": declare("kv_extend", [P, I64, I64, P, P, I64, P, P, I64, I32, I64, P, P, P, P, P, P]),
               "kv_release": declare("kv_release", [P, I64, I64, P, P, I64, P, P, I64, I32, P, P, P]),
               "kv_append": declare("kv_append", [P, I64, I32, I32, I32, P, I64, I64, P, I64, I64, P, I64, P]),
               "kv_read": declare("kv_read", [P, I64, I32, I32, I32, P, I64, P, P, P]),
               "kv_attention_workspace_bytes": declare("kv_attention_workspace_bytes",
                                                       [I64, I32, I32, I32, I64, I64, I32, I32, I64, I64], SZ),
               "kv_attention": declare("kv_attention", [P, I64, I64, I64, I32, P, I64, I32, I32, I32, P, I64, I64, P, P, I64, I64,
                                                        F32, I64, P, P, P, SZ, P])}
        _fn.update(got)
    return _fn


# ------------------------------------------------------------ C ABI mirror

def kv_extend(table, ld_table, table_width, lengths, counts, requests, free, free_count, pages, page_size, tokens, offsets,
              lengths_out, slots, positions, free_count_out, stream=None):
    _check(_functions()["kv_extend"](_p(table), ld_table, table_width, _p(lengths), _p(counts), requests, _p(free),
                                     _p(free_count), pages, page_size, tokens, _p(offsets), _p(lengths_out), _p(slots),
                                     _p(positions), _p(free_count_out), _s(stream)), "kv_extend")


def kv_release(table, ld_table, table_width, lengths, finished, requests, free, free_count, pages, page_size, lengths_out,
               free_count_out, stream=None):
    _check(_functions()["kv_release"](_p(table), ld_table, table_width, _p(lengths), _p(finished), requests, _p(free),
                                      _p(free_count), pages, page_size, _p(lengths_out), _p(free_count_out), _s(stream)),
           "kv_release")


def kv_append(cache, pages, page_size, kv_heads, head_dim, k, k_token, k_head, v, v_token, v_head, slots, tokens, stream=None):
    _check(_functions()["kv_append"](_p(cache), pages, page_size, kv_heads, head_dim, _p(k), k_token, k_head, _p(v), v_token,
                                     v_head, _p(slots), tokens, _s(stream)), "kv_append")


def kv_read(cache, pages, page_size, kv_heads, head_dim, slots, tokens, k, v, stream=None):
    _check(_functions()["kv_read"](_p(cache), pages, page_size, kv_heads, head_dim, _p(slots), tokens, _p(k), _p(v),
                                   _s(stream)), "kv_read")


def kv_attention_workspace_bytes(tokens, heads, kv_heads, head_dim, sequences, table_width, page_size, ragged, max_queries,
                                 window):
    return _functions()["kv_attention_workspace_bytes"](tokens, heads, kv_heads, head_dim, sequences, table_width, page_size,
                                                        ragged, max_queries, window)


def kv_attention(q, q_token, q_head, tokens, heads, cache, pages, page_size, kv_heads, head_dim, table, ld_table, table_width,
                 lengths, offsets, sequences, max_queries, scale, window, out, lse=None, workspace=None, workspace_bytes=0,
                 stream=None):
    _check(_functions()["kv_attention"](_p(q), q_token, q_head, tokens, heads, _p(cache), pages, page_size, kv_heads, head_dim,
                                        _p(table), ld_table, table_width, _p(lengths), _p(offsets), sequences, max_queries,
                                        scale, window, _p(out), _p(lse), _p(workspace), workspace_bytes, _s(stream)),
           "kv_attention")


# ------------------------------------------------------------------ operators

_ops = None


def _load():
    global _ops
    _ops = extension()
    return _ops


def new(pages, page_size, kv_heads, head_dim, device=None):
    """An empty cache, uint8 [pages, kv_heads, page_size * (head_dim + head_dim / 16)]:
    of every token and head the MXFP4 codes and scales of a key and a value.
    page_size 16, 32, 64, 128 or 256; head_dim 64, 128 or 256.  Calls read the page
    size off the cache's shape."""
    if page_size not in (16, 32, 64, 128, 256):
        raise ValueError("page_size must be 16, 32, 64, 128 or 256")
    if head_dim not in (64, 128, 256):
        raise ValueError("head_dim must be 64, 128 or 256")
    if pages < 1 or kv_heads < 1:
        raise ValueError("a cache has at least one page and one head")
    return torch.zeros((pages, kv_heads, page_size * (head_dim + head_dim // 16)), dtype=torch.uint8, device=device)


def pool(pages, device=None):
    """(free, free_count) of a cache without requests: the stack of its pages (int32
    [pages], page 0 on top) and their number (int32 [1])."""
    free = torch.arange(pages - 1, -1, -1, dtype=torch.int32, device=device)
    return free, torch.full((1,), pages, dtype=torch.int32, device=device)


class Extension(NamedTuple):
    """Of B requests with new tokens, ``tokens`` rows at most: the rows of each
    request int32 [B + 1], its length with them [B], the slot (-1: none) and the
    position of each row [tokens], and the number of free pages left [1]."""
    offsets: torch.Tensor
    lengths: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    free_count: torch.Tensor


_new_tuple = tuple.__new__


def extend(table, lengths, counts, free, free_count, tokens, page_size, stream=None):
    """Pages for counts[b] new tokens behind the lengths[b] of each request b (all
    int32 [B]), from the end of the stack ``free`` (int32 [pages], of which
    free_count (int32 [1]) are left), written to table (int32 [B, W], in place) behind
    those the request has.  tokens: rows to return slots and positions for; rows
    behind the last request's get slot -1.  A request whose pages are not to be had
    (the stack is empty, the table or the rows too short) gets nothing: its length
    stays and its rows have slot -1."""
    if stream is not None:
        return on_stream(stream, (table, lengths, counts, free, free_count),
                         lambda: extend(table, lengths, counts, free, free_count, tokens, page_size))
    return _new_tuple(Extension, (_ops or _load()).extend(table, lengths, counts, free, free_count, tokens, page_size))


def release(table, lengths, finished, free, free_count, page_size, stream=None):
    """Give back the pages of the requests with ``finished`` (bool [B]): they go on the
    stack ``free`` in place, their entries of the table become -1.  Returns (lengths,
    free_count), the lengths of finished requests 0."""
    if stream is not None:
        return on_stream(stream, (table, lengths, finished, free, free_count),
                         lambda: release(table, lengths, finished, free, free_count, page_size))
    return (_ops or _load()).release(table, lengths, finished, free, free_count, page_size)


def append(cache, k, v, slots, stream=None):
    """Write k and v (BF16 [T, kv_heads, head_dim], unit stride along the head) to
    their slots (int32 [T], different ones; outside the cache: skipped) as MXFP4 with
    blocks of 32 along the head, with the scales and codes of ``mxfp4.quantize``."""
    if stream is not None:
        return on_stream(stream, (cache, k, v, slots), lambda: append(cache, k, v, slots))
    return (_ops or _load()).append(cache, k, v, slots)


def read(cache, slots, head_dim, stream=None):
    """(k, v) BF16 [T, kv_heads, head_dim] at slots (int32 [T]); zeros outside the
    cache."""
    if stream is not None:
        return on_stream(stream, (cache, slots), lambda: read(cache, slots, head_dim))
    return (_ops or _load()).read(cache, slots, head_dim)


def attention(q, cache, table, lengths, offsets=None, scale=None, window=0, max_queries=None, lse=False, out=None, stream=None):
    """softmax(scale q k^T) v in BF16 [T, heads, head_dim] for q (BF16, unit stride
    along the head) over the keys that table (int32 [B, W]) and lengths (int32 [B])
    give each sequence.  The queries of sequence b, rows offsets[b] .. offsets[b + 1] -
    1 (int32 [B + 1]; None: one each), stand at the end of its lengths[b] keys: each sees
    the keys up to its own, with window > 0 the last ``window`` of them; keys that the
    table does not hold are not there, also behind its last page.  heads is a multiple of
    the cache's, whose head h serves heads h * group .. + group - 1.  scale: head_dim **
    -0.5 unless given.  max_queries: the longest run of queries, where the program
    knows it (without it a decoding step of several sequences with offsets is taken for a
    prompt, whose kernel answers single tokens more slowly); it decides how the work is
    cut, not what comes out.  lse=True: (out, log of the
    softmax's sum fp32 [T, heads]), to join parts.  Queries without a key get zeros (and
    -inf); rows of no sequence are not written.  out: dense, apart from q and the
    cache."""
    if stream is not None:
        return on_stream(stream, (q, cache, table, lengths, offsets, out),
                         lambda: attention(q, cache, table, lengths, offsets, scale, window, max_queries, lse, out))
    return (_ops or _load()).attention(q, cache, table, lengths, offsets, scale, window, max_queries, lse, out)
