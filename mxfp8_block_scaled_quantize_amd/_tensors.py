"""The extension module of the tensor-level operators, their C functions and
their use on another stream."""

from __future__ import annotations

import ctypes

import torch
from torch.autograd import forward_ad

from . import lib


def declare(name, argtypes, restype=ctypes.c_int):
    """The C function `name` of libmxfp8 with its argument types set."""
    f = getattr(lib(), name)
    f.restype = restype
    f.argtypes = argtypes
    return f


def extension():
    """The module _mx_torch; raises if it has not been built."""
    try:
        from . import _mx_torch
    except ImportError as e:
        raise RuntimeError("_mx_torch.so is not built (run mxfp8_block_scaled_quantize_amd.build.build()): %s" % e) from e
    return _mx_torch


def on_stream(stream, tensors, call):
    """Run `call` with `stream` (a torch stream or a raw handle, of the tensors'
    device) current: its outputs belong to that stream, and its inputs' memory is
    not handed out again before the stream is done."""
    device = next((t.device for t in tensors if getattr(t, "is_cuda", False)), None)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    elif device is not None and stream.device != device:
        raise ValueError("stream is on %s, the tensors on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        result = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return result


def no_tangent(where, *tensors):
    """Refuse dual tensors: the layers have no forward-mode derivative, and a
    tangent must not get lost on a path without autograd."""
    if forward_ad._current_level < 0:
        return
    for t in tensors:
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("%s does not propagate forward-mode tangents" % where)
