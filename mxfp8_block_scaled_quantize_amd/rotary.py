"""Rotary positions: queries and keys turned by angles that grow with their position.

``turns`` gives the frequencies of a head's pairs, plain or stretched for contexts
longer than a model was trained on; ``rotate`` turns q and k with them, in one
launch, differentiably.  The kernel is that of ``include/rotary.h``
(``rotary_rotate`` mirrors it); there is no fallback.
"""

from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _p, _s
from ._tensors import declare, extension, on_stream

ROTARY_FP32, ROTARY_BF16, ROTARY_FP16 = 0, 1, 2
ROTARY_INTERLEAVED = 1
ROTARY_INVERSE = 2

EXPORTED = ("rotary_rotate",)

_fn = {}


def _functions():
    if not _fn:
        P, I64, I32, U32, F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_float
        _fn["rotary_rotate"] = declare("rotary_rotate", [P, I64, I64, I64, P, I64, I64, I64, I32, I64, I64, I64, P, P, F32, U32,
                                                         P, P, P])
    return _fn


# ------------------------------------------------------------ C ABI mirror

def rotary_rotate(q, q_token, q_head, q_heads, k, k_token, k_head, k_heads, dtype, tokens, head_dim, pairs, positions, turns,
                  magnitude, flags, q_out, k_out=None, stream=None):
    _check(_functions()["rotary_rotate"](_p(q), q_token, q_head, q_heads, _p(k), k_token, k_head, k_heads, dtype, tokens,
                                         head_dim, pairs, _p(positions), _p(turns), magnitude, flags, _p(q_out), _p(k_out),
                                         _s(stream)), "rotary_rotate")


# ------------------------------------------------------------------ operators

def turns(dims, base=10000.0, scaling=None, factor=1.0, trained=None, fast=32.0, slow=1.0, low=1.0, high=4.0, device=None):
    """(turns per position fp64 [dims / 2], magnitude) for the first ``dims`` dimensions
    of a head: base ** (-2 f / dims) / (2 pi), and 1.

    scaling, for contexts ``factor`` times as long as the ``trained`` ones:
      "linear"  every frequency divided by factor;
      "ntk"     the base times factor ** (dims / (dims - 2)): the fastest pair stays, the
                slowest is divided by factor;
      "yarn"    pairs that turn ``fast`` times or more in ``trained`` positions stay,
                those that turn ``slow`` times or less are divided by factor, in between
                by pair number, linearly; magnitude 0.1 ln(factor) + 1;
      "bands"   the same with the border by wavelength: pairs that turn ``high`` times
                or more stay, ``low`` times or less are divided, in between linearly in
                the number of turns; magnitude 1."""
    if dims < 2 or dims % 2:
        raise ValueError("dims must be even and at least 2")
    if base <= 1 or factor < 1:
        raise ValueError("base must be over 1 and factor at least 1")
    n = dims // 2
    f = torch.arange(n, dtype=torch.float64)
    magnitude = 1.0
    if scaling == "ntk":
        if dims < 4:
            raise ValueError("scaling 'ntk' needs at least two pairs")
        base = base * factor ** (dims / (dims - 2))
    t = float(base) ** (-f / n) / (2 * math.pi)
    if scaling == "linear":
        t = t / factor
    elif scaling in ("yarn", "bands"):
        if trained is None or trained < 1:
            raise ValueError("scaling %r needs the trained length" % scaling)
        if scaling == "yarn":
            def pair_of(rounds):   # the pair that turns so often in the trained length
                return n * math.log(trained / (rounds * 2 * math.pi)) / math.log(base)
            first, last = max(math.floor(pair_of(fast)), 0), min(math.ceil(pair_of(slow)), dims - 1)
            stretched = ((f - first) / max(last - first, 1e-3)).clamp(0, 1)
            magnitude = 0.1 * math.log(factor) + 1.0
        else:
            if high <= low:
                raise ValueError("high must be over low")
            stretched = 1 - ((t * trained - low) / (high - low)).clamp(0, 1)
        t = t * (1 - stretched) + t / factor * stretched
    elif scaling not in (None, "ntk"):
        raise ValueError("scaling must be None, 'linear', 'ntk', 'yarn' or 'bands'")
    return t.to(device), magnitude


_ops = None


def _load():
    global _ops
    _ops = extension()
    return _ops


def rotate(q, k, positions, turns, interleaved=False, magnitude=1.0, stream=None):
    """(q, k), or q with k=None, turned: q and k [T, heads, head_dim] (fp32, BF16 or
    FP16, unit stride along the head), positions int32 [T], turns fp64 [pairs].  The
    first 2 * pairs dimensions of a head are pairs (f, f + pairs), or (2 f, 2 f + 1) with
    interleaved=True; each is turned by position * turns[f] whole turns and multiplied
    by magnitude; the others are copied.  Differentiable in q and k."""
    if stream is not None:
        return on_stream(stream, (q, k, positions, turns), lambda: rotate(q, k, positions, turns, interleaved, magnitude))
    return (_ops or _load()).rotate(q, k, positions, turns, interleaved, magnitude)
