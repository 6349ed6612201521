"""MXFP4 (E2M1 codes, one E8M0 scale per 32 values): quantize, dequantize and
the block-scaled products, dense and grouped.

``mxfp4_*`` mirror the C ABI of ``include/mxfp4.h``; ``quantize``,
``dequantize``, ``gemm`` and ``grouped_gemm`` check their tensors, allocate the
outputs and call it (in the extension module ``_mx_torch``).  Codes are uint8, two to a byte (lower index in the low nibble);
packed scale words are int32 [K / 128, rows], as for MXFP8.  Every step runs in
the HIP kernels of ``libmxfp8.so``; there is no fallback.  A tensor passed as
``out`` counts as modified in place; one that requires a gradient is refused
while gradients are enabled.
"""

from __future__ import annotations

import ctypes

from . import _check, _p, _s
from ._tensors import declare, extension, on_stream

MXFP4_ROWWISE = 1
MXFP4_COLWISE = 2
MXFP4_PACKED_SCALES = 16
MXFP4_GEMM_ACCUMULATE = 1
MXFP4_GEMM_SWIGLU = 8

EXPORTED = ("mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_grouped_gemm")

_fn = {}


def _functions():
    if not _fn:
        P, I64, I32, U32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
        got = {"mxfp4_quantize": declare("mxfp4_quantize", [P, I64, I64, I64, I64, P, U32, P, P, P, P, P]),
               "mxfp4_dequantize": declare("mxfp4_dequantize", [P, P, I64, I64, P, I64, U32, P]),
               "mxfp4_gemm": declare("mxfp4_gemm", [P, P, P, P, P, I64, I64, I64, I64, U32, P]),
               "mxfp4_grouped_gemm": declare("mxfp4_grouped_gemm",
                                             [P, P, P, P, P, I32, P, I64, I64, I64, I64, U32, P])}
        _fn.update(got)
    return _fn


# ------------------------------------------------------------ C ABI mirror

def mxfp4_quantize(x, x_rows, rows, cols, ld_x, index, flags, q_row=None, s_row=None, q_colT=None, s_colT=None,
                   stream=None):
    _check(_functions()["mxfp4_quantize"](_p(x), x_rows, rows, cols, ld_x, _p(index), flags, _p(q_row), _p(s_row), _p(q_colT),
                                          _p(s_colT), _s(stream)), "mxfp4_quantize")


def mxfp4_dequantize(q, s, rows, cols, out, ld_out, flags, stream=None):
    _check(_functions()["mxfp4_dequantize"](_p(q), _p(s), rows, cols, _p(out), ld_out, flags, _s(stream)),
           "mxfp4_dequantize")


def mxfp4_gemm(a, a_packed, b, b_packed, c, ldc, M, N, K, flags, stream=None):
    _check(_functions()["mxfp4_gemm"](_p(a), _p(a_packed), _p(b), _p(b_packed), _p(c), ldc, M, N, K, flags, _s(stream)),
           "mxfp4_gemm")


def mxfp4_grouped_gemm(a, a_packed, b, b_packed, offsets, G, c, ldc, M_total, N, K, flags, stream=None):
    _check(_functions()["mxfp4_grouped_gemm"](_p(a), _p(a_packed), _p(b), _p(b_packed), _p(offsets), G, _p(c), ldc, M_total, N,
                                              K, flags, _s(stream)), "mxfp4_grouped_gemm")


# ------------------------------------------------------ allocating helpers

_ops = None


def _load():
    global _ops
    _ops = extension()
    return _ops


def quantize(x, rowwise=True, colwise=False, packed=False, index=None, stream=None):
    """MXFP4 copies of a BF16 [R, C] tensor (unit column stride) as a dict.

    rowwise: "q_row" uint8 [R, C / 2] and "s_row" uint8 [R, C / 32], or with
    packed=True "p_row" int32 [C / 128, R]; colwise: the transposed copy,
    "q_colT" uint8 [C, R / 2] and "s_colT" [C, R / 32] or "p_colT" int32
    [R / 128, C].  index (int32 [n], rowwise alone): row r of the copy is x's
    row index[r] (n rows; zeros for an index outside x), as the tokens of
    ``moe.dispatch`` name them."""
    if stream is not None:
        return on_stream(stream, (x, index), lambda: quantize(x, rowwise, colwise, packed, index))
    return (_ops or _load()).quantize(x, rowwise, colwise, packed, index)


def dequantize(q, scales, out=None, stream=None):
    """BF16 [R, K] values of codes q [R, K / 2] with packed scale words int32
    [K / 128, R] or scale bytes uint8 [R, K / 32]."""
    if stream is not None:
        return on_stream(stream, (q, scales, out), lambda: dequantize(q, scales, out))
    return (_ops or _load()).dequantize(q, scales, out)


def gemm(a, a_packed, b, b_packed, out=None, accumulate=False, swiglu=False, stream=None):
    """C = dq(A) dq(B)^T in BF16 for codes a [M, K / 2], b [N, K / 2] and their
    packed scale words.  accumulate=True adds the product to ``out``;
    swiglu=True: b is [2N, K / 2] (gate rows, then up rows) and C [M, N] =
    SiLU(gate product) * up product."""
    if stream is not None:
        return on_stream(stream, (a, a_packed, b, b_packed, out),
                         lambda: gemm(a, a_packed, b, b_packed, out, accumulate, swiglu))
    return (_ops or _load()).gemm(a, a_packed, b, b_packed, out, accumulate, swiglu)


def grouped_gemm(a, a_packed, b, b_packed, offsets, out=None, accumulate=False, swiglu=False, stream=None):
    """Ragged grouped product: rows offsets[g] .. offsets[g + 1] - 1 of a (int32
    offsets on the device) times expert g of b [G, N, K / 2] (b_packed [K / 128,
    G * N]); swiglu=True: experts of 2N rows, C [M, N].  Rows outside every
    group are not written."""
    if stream is not None:
        return on_stream(stream, (a, a_packed, b, b_packed, offsets, out),
                         lambda: grouped_gemm(a, a_packed, b, b_packed, offsets, out, accumulate, swiglu))
    return (_ops or _load()).grouped_gemm(a, a_packed, b, b_packed, offsets, out, accumulate, swiglu)
