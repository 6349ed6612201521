"""Mixture-of-experts operators: routing, dispatch and combination.

``route`` chooses the experts of every token and their weights (differentiable
in the logits), ``dispatch`` sorts the (token, slot) pairs by expert, and
``combine`` adds up the experts' outputs by the weights (differentiable in
both).  Between them stand the grouped products, on rows gathered by
``dispatch``'s tokens (``mxfp4.quantize(x, index=token, packed=True)``).  The
kernels are those of ``include/moe.h``; there is no fallback.
"""

from __future__ import annotations

import ctypes
from typing import NamedTuple

import torch

from ._tensors import check, declare, launch, need, on_stream

MOE_FP32, MOE_BF16, MOE_FP16 = 0, 1, 2
MOE_ROUTE_SIGMOID = 1
MOE_ROUTE_RENORMALIZE = 2
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOP_K = 64

EXPORTED = ("moe_route", "moe_route_backward", "moe_dispatch_workspace_bytes", "moe_dispatch", "moe_combine",
            "moe_combine_backward")

_DTYPES = {torch.float32: MOE_FP32, torch.bfloat16: MOE_BF16, torch.float16: MOE_FP16}

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


def _address(t):
    return None if t is None else t if isinstance(t, int) else t.data_ptr()


def _stream(stream):
    if isinstance(stream, int):
        return stream
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


# ------------------------------------------------------------ C ABI mirror

def moe_route(logits, dtype, tokens, experts, ld, bias, top_k, groups, top_groups, group_top, flags, weights, ids,
              stream=None):
    p = _address
    check(_functions()["moe_route"](p(logits), dtype, tokens, experts, ld, p(bias), top_k, groups, top_groups, group_top,
                                    flags, p(weights), p(ids), _stream(stream)), "moe_route")


def moe_route_backward(logits, dtype, tokens, experts, ld, ids, dweights, top_k, flags, dlogits, stream=None):
    p = _address
    check(_functions()["moe_route_backward"](p(logits), dtype, tokens, experts, ld, p(ids), p(dweights), top_k, flags,
                                             p(dlogits), _stream(stream)), "moe_route_backward")


def moe_dispatch_workspace_bytes(tokens, experts, top_k):
    return _functions()["moe_dispatch_workspace_bytes"](tokens, experts, top_k)


def moe_dispatch(ids, tokens, experts, top_k, offsets, token, position, workspace=None, workspace_bytes=0, stream=None):
    p = _address
    check(_functions()["moe_dispatch"](p(ids), tokens, experts, top_k, p(offsets), p(token), p(position), p(workspace),
                                       workspace_bytes, _stream(stream)), "moe_dispatch")


def moe_combine(y, dtype, rows, ld_y, position, weights, tokens, top_k, hidden, out, stream=None):
    p = _address
    check(_functions()["moe_combine"](p(y), dtype, rows, ld_y, p(position), p(weights), tokens, top_k, hidden, p(out),
                                      _stream(stream)), "moe_combine")


def moe_combine_backward(y, dtype, rows, ld_y, position, weights, tokens, top_k, hidden, dout, ld_dout, dy, dweights,
                         workspace=None, workspace_bytes=0, stream=None):
    p = _address
    check(_functions()["moe_combine_backward"](p(y), dtype, rows, ld_y, p(position), p(weights), tokens, top_k, hidden,
                                               p(dout), ld_dout, p(dy), p(dweights), p(workspace), workspace_bytes,
                                               _stream(stream)), "moe_combine_backward")


# ------------------------------------------------------------------- routing

def _route(logits, bias, top_k, groups, top_groups, group_top, flags):
    T, E = logits.shape
    dev = logits.device
    weights = torch.empty((T, top_k), dtype=torch.float32, device=dev)
    ids = torch.empty((T, top_k), dtype=torch.int32, device=dev)
    launch(_functions()["moe_route"], "moe_route", dev, logits.data_ptr(), _DTYPES[logits.dtype], T, E,
           max(logits.stride(0), E), None if bias is None else bias.data_ptr(), top_k, groups, top_groups, group_top,
           flags, weights.data_ptr(), ids.data_ptr())
    return weights, ids


class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, bias, top_k, groups, top_groups, group_top, flags):
        weights, ids = _route(logits, bias, top_k, groups, top_groups, group_top, flags)
        ctx.save_for_backward(logits, ids)
        ctx.flags = flags
        ctx.mark_non_differentiable(ids)
        ctx.set_materialize_grads(False)
        return weights, ids

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dweights, _):
        if dweights is None:
            return (None,) * 7
        logits, ids = ctx.saved_tensors
        T, E = logits.shape
        if dweights.dtype is not torch.float32 or not dweights.is_contiguous():
            dweights = dweights.float().contiguous()
        d = torch.empty((T, E), dtype=logits.dtype, device=logits.device)
        launch(_functions()["moe_route_backward"], "moe_route_backward", logits.device, logits.data_ptr(),
               _DTYPES[logits.dtype], T, E, max(logits.stride(0), E), ids.data_ptr(), dweights.data_ptr(), ids.shape[1],
               ctx.flags, d.data_ptr())
        return d, None, None, None, None, None, None


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
    if not isinstance(logits, torch.Tensor) or logits.dtype not in _DTYPES or logits.dim() != 2:
        raise ValueError("logits must be a [tokens, experts] tensor of float32, bfloat16 or float16")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA (HIP) tensor, got %s" % logits.device)
    if logits.stride(1) != 1:
        raise ValueError("logits must have unit stride along the experts")
    if scores == "softmax":
        flags = 0
    elif scores == "sigmoid":
        flags = MOE_ROUTE_SIGMOID
    else:
        raise ValueError("scores must be 'softmax' or 'sigmoid'")
    if renormalize:
        flags |= MOE_ROUTE_RENORMALIZE
    if top_k < 1:
        raise ValueError("top_k must be at least 1")
    if bias is not None:
        need(bias, "bias", torch.float32, (logits.shape[1],), logits.device)
    if logits.requires_grad and torch.is_grad_enabled():
        return _Route.apply(logits, bias, top_k, groups, top_groups, group_top, flags)
    return _route(logits, bias, top_k, groups, top_groups, group_top, flags)


# ------------------------------------------------------------------ dispatch

class Dispatch(NamedTuple):
    """offsets int32 [E + 1] of the experts' rows, the token of each row int32
    [T * K] (-1 behind the last expert's) and the row of each slot int32 [T, K]
    (-1 for an id outside the experts)."""
    offsets: torch.Tensor
    token: torch.Tensor
    position: torch.Tensor


def dispatch(ids, experts, stream=None):
    """Stable counting sort of the slots of ids (int32 [T, K]) by expert."""
    if stream is not None:
        return on_stream(stream, (ids,), lambda: dispatch(ids, experts))
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be an int32 [tokens, top_k] tensor")
    T, K = ids.shape
    need(ids, "ids", torch.int32, (T, K))
    dev = ids.device
    f = _functions()
    offsets = torch.empty((experts + 1,), dtype=torch.int32, device=dev)
    token = torch.empty((T * K,), dtype=torch.int32, device=dev)
    position = torch.empty((T, K), dtype=torch.int32, device=dev)
    n = f["moe_dispatch_workspace_bytes"](T, experts, K)
    work = torch.empty((n // 4,), dtype=torch.int32, device=dev) if n else None
    launch(f["moe_dispatch"], "moe_dispatch", dev, ids.data_ptr(), T, experts, K, offsets.data_ptr(), token.data_ptr(),
           position.data_ptr(), _address(work), n)
    return Dispatch(offsets, token, position)


# ------------------------------------------------------------------- combine

def _combine(y, position, weights):
    rows, H = y.shape
    T, K = position.shape
    out = torch.empty((T, H), dtype=y.dtype, device=y.device)
    launch(_functions()["moe_combine"], "moe_combine", y.device, y.data_ptr(), _DTYPES[y.dtype], rows,
           max(y.stride(0), H), position.data_ptr(), weights.data_ptr(), T, K, H, out.data_ptr())
    return out


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, position, weights):
        ctx.save_for_backward(y, position, weights)
        return _combine(y, position, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        y, position, weights = ctx.saved_tensors
        rows, H = y.shape
        T, K = position.shape
        dev = y.device
        if dout.stride(1) != 1 or dout.stride(0) < H:   # expanded or transposed gradients
            dout = dout.contiguous()
        dy = dw = work = None
        if ctx.needs_input_grad[0]:
            dy = torch.empty((rows, H), dtype=y.dtype, device=dev)
            work = torch.empty((rows,), dtype=torch.int32, device=dev)
        if ctx.needs_input_grad[2]:
            dw = torch.empty((T, K), dtype=torch.float32, device=dev)
        launch(_functions()["moe_combine_backward"], "moe_combine_backward", dev, y.data_ptr(), _DTYPES[y.dtype], rows,
               max(y.stride(0), H), position.data_ptr(), weights.data_ptr(), T, K, H, dout.data_ptr(), dout.stride(0),
               _address(dy), _address(dw), _address(work), 0 if work is None else 4 * rows)
        return dy, None, dw


def combine(y, position, weights, stream=None):
    """out[t] = sum_k weights[t, k] * y[position[t, k]] for y [rows, H] (fp32,
    BF16 or FP16, unit column stride), position int32 [T, K] and weights fp32
    [T, K]; out has y's type, sums are fp32.  A position outside y (-1) adds
    nothing.  Differentiable in y and weights."""
    if stream is not None:
        return on_stream(stream, (y, position, weights), lambda: combine(y, position, weights))
    if not isinstance(y, torch.Tensor) or y.dtype not in _DTYPES or y.dim() != 2 or y.stride(1) != 1:
        raise ValueError("y must be a [rows, hidden] tensor of float32, bfloat16 or float16 with unit column stride")
    if not y.is_cuda:
        raise ValueError("y must be a CUDA (HIP) tensor, got %s" % y.device)
    if not isinstance(position, torch.Tensor) or position.dim() != 2:
        raise ValueError("position must be an int32 [tokens, top_k] tensor")
    need(position, "position", torch.int32, position.shape, y.device)
    need(weights, "weights", torch.float32, position.shape, y.device)
    if torch.is_grad_enabled() and (y.requires_grad or weights.requires_grad):
        return _Combine.apply(y, position, weights)
    return _combine(y, position, weights)
