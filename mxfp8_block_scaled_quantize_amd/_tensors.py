"""Argument checks and stream handling shared by the tensor-level operators."""

from __future__ import annotations

import torch

from . import MXFP8Error, lib


def declare(name, argtypes, restype=None):
    """The C function `name` of libmxfp8 with its argument types set."""
    import ctypes
    f = getattr(lib(), name)
    f.restype = ctypes.c_int if restype is None else restype
    f.argtypes = argtypes
    return f


def check(status, where):
    if status != 0:
        raise MXFP8Error(status, where)


def need(t, name, dtype, shape, device=None):
    """A dense GPU tensor of this type and shape (on `device`, when given)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA (HIP) tensor, got %s" % (name, t.device))
    if t.dtype is not dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def launch(f, where, device, *args):
    """Call a C entry point with the current stream of `device` (its last
    argument), that device being current during the call."""
    index = device.index
    if torch._C._cuda_getDevice() == index:
        status = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != 0:
        raise MXFP8Error(status, where)


def on_stream(stream, tensors, call):
    """Run `call` with `stream` current: its outputs belong to that stream, and
    its inputs' memory is not handed out again before the stream is done."""
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream)
    with torch.cuda.stream(stream):
        result = call()
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return result
