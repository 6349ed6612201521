"""Mixture-of-experts operators: routing, dispatch and combination.

``route`` chooses the experts of every token and their weights (differentiable
in the logits), ``dispatch`` sorts the (token, slot) pairs by expert, and
``combine`` adds up the experts' outputs by the weights (differentiable in
both).  Between them stand the grouped products, on rows gathered by
``dispatch``'s tokens (``mxfp4.quantize(x, index=token, packed=True)``).  The
kernels are those of ``include/moe.h`` (``moe_*`` mirror it); there is no
fallback.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from . import _check, _p, _s
from ._tensors import declare, extension, on_stream

MOE_FP32, MOE_BF16, MOE_FP16 = 0, 1, 2
MOE_ROUTE_SIGMOID = 1
MOE_ROUTE_RENORMALIZE = 2
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOP_K = 64

EXPORTED = ("moe_route", "moe_route_backward", "moe_dispatch_workspace_bytes", "moe_dispatch", "moe_combine",
            "moe_combine_backward")

_fn = {}


def _functions():
    if not _fn:
        P, I64, I32, U32, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        got = {"moe_route": declare("moe_route", [P, I32, I64, I64, I64, P, I32, I32, I32, I32, U32, P, P, P]),
               "moe_route_backward": declare("moe_route_backward", [P, I32, I64, I64, I64, P, P, I32, U32, P, P]),
               "moe_dispatch_workspace_bytes": declare("moe_dispatch_workspace_bytes", [I64, I64, I64], SZ),
               "moe_dispatch": declare("moe_dispatch", [P, I64, I64, I64, P, P, P, P, SZ, P]),
               "moe_combine": declare("moe_combine", [P, I32, I64, I64, P, P, I64, I64, I64, P, P]),
               "moe_combine_backward": declare("moe_combine_backward", [P, I32, I64, I64, P, P, I64, I64, I64, P, I64, P,
                                                                        P, P, SZ, P])}
        _fn.update(got)
    return _fn


# ------------------------------------------------------------ C ABI mirror

def moe_route(logits, dtype, tokens, experts, ld, bias, top_k, groups, top_groups, group_top, flags, weights, ids,
              stream=None):
    _check(_functions()["moe_route"](_p(logits), dtype, tokens, experts, ld, _p(bias), top_k, groups, top_groups, group_top,
                                     flags, _p(weights), _p(ids), _s(stream)), "moe_route")


def moe_route_backward(logits, dtype, tokens, experts, ld, ids, dweights, top_k, flags, dlogits, stream=None):
    _check(_functions()["moe_route_backward"](_p(logits), dtype, tokens, experts, ld, _p(ids), _p(dweights), top_k, flags,
                                              _p(dlogits), _s(stream)), "moe_route_backward")


def moe_dispatch_workspace_bytes(tokens, experts, top_k):
    return _functions()["moe_dispatch_workspace_bytes"](tokens, experts, top_k)


def moe_dispatch(ids, tokens, experts, top_k, offsets, token, position, workspace=None, workspace_bytes=0, stream=None):
    _check(_functions()["moe_dispatch"](_p(ids), tokens, experts, top_k, _p(offsets), _p(token), _p(position), _p(workspace),
                                        workspace_bytes, _s(stream)), "moe_dispatch")


def moe_combine(y, dtype, rows, ld_y, position, weights, tokens, top_k, hidden, out, stream=None):
    _check(_functions()["moe_combine"](_p(y), dtype, rows, ld_y, _p(position), _p(weights), tokens, top_k, hidden, _p(out),
                                       _s(stream)), "moe_combine")


def moe_combine_backward(y, dtype, rows, ld_y, position, weights, tokens, top_k, hidden, dout, ld_dout, dy, dweights,
                         workspace=None, workspace_bytes=0, stream=None):
    _check(_functions()["moe_combine_backward"](_p(y), dtype, rows, ld_y, _p(position), _p(weights), tokens, top_k, hidden,
                                                _p(dout), ld_dout, _p(dy), _p(dweights), _p(workspace), workspace_bytes,
                                                _s(stream)), "moe_combine_backward")


# ------------------------------------------------------------------ operators

_ops = None


def _load():
    global _ops
    _ops = extension()
    return _ops


_SCORES = {"softmax": 0, "sigmoid": MOE_ROUTE_SIGMOID}


def route(logits, top_k, scores="softmax", bias=None, groups=1, top_groups=1, group_top=2, renormalize=True, stream=None):
    """(weights fp32 [T, top_k], expert ids int32 [T, top_k]) for router logits
    [T, E] (fp32, BF16 or FP16, unit column stride), the largest choice first.

    scores: "softmax" over the E experts or "sigmoid" of each.  bias (fp32 [E])
    is added for the choice alone, not to the weights.  groups > 1: the experts
    stand in ``groups`` equal runs, and only those of the ``top_groups`` runs
    with the largest sums of their ``group_top`` (1 or 2) best choices can be
    chosen.  renormalize: weights divided by their sum.  Ties go to the lowest
    index.  The weights are differentiable in the logits (the choice is a
    constant; bias has no gradient)."""
    if stream is not None:
        return on_stream(stream, (logits, bias),
                         lambda: route(logits, top_k, scores, bias, groups, top_groups, group_top, renormalize))
    if scores not in _SCORES:
        raise ValueError("scores must be 'softmax' or 'sigmoid'")
    flags = _SCORES[scores] | (MOE_ROUTE_RENORMALIZE if renormalize else 0)
    return (_ops or _load()).route(logits, top_k, flags, bias, groups, top_groups, group_top)


class Dispatch(NamedTuple):
    """offsets int32 [E + 1] of the experts' rows, the token of each row int32
    [T * K] (-1 behind the last expert's) and the row of each slot int32 [T, K]
    (-1 for an id outside the experts)."""
    offsets: torch.Tensor
    token: torch.Tensor
    position: torch.Tensor


_new_tuple = tuple.__new__


def dispatch(ids, experts, stream=None):
    """Stable counting sort of the slots of ids (int32 [T, K]) by expert."""
    if stream is not None:
        return on_stream(stream, (ids,), lambda: dispatch(ids, experts))
    return _new_tuple(Dispatch, (_ops or _load()).dispatch(ids, experts))


def combine(y, position, weights, stream=None):
    """out[t] = sum_k weights[t, k] * y[position[t, k]] for y [rows, H] (fp32,
    BF16 or FP16, unit column stride), position int32 [T, K] and weights fp32
    [T, K]; out has y's type, sums are fp32.  A position outside y (-1) adds
    nothing.  Differentiable in y and weights."""
    if stream is not None:
        return on_stream(stream, (y, position, weights), lambda: combine(y, position, weights))
    return (_ops or _load()).combine(y, position, weights)
