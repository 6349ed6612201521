"""MXFP4 (E2M1 codes, one E8M0 scale per 32 values): quantize, dequantize and
the block-scaled products, dense and grouped.

``mxfp4_*`` mirror the C ABI of ``include/mxfp4.h``; ``quantize``,
``dequantize``, ``gemm`` and ``grouped_gemm`` allocate outputs with torch and
call them.  Codes are uint8, two to a byte (lower index in the low nibble);
packed scale words are int32 [K / 128, rows], as for MXFP8.  Every step runs in
the HIP kernels of ``libmxfp8.so``; there is no fallback.
"""

from __future__ import annotations

import ctypes

import torch

from ._tensors import check, declare, launch, need, on_stream

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


def _address(t):
    return None if t is None else t if isinstance(t, int) else t.data_ptr()


def _stream(stream):
    if isinstance(stream, int):
        return stream
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


# ------------------------------------------------------------ C ABI mirror

def mxfp4_quantize(x, x_rows, rows, cols, ld_x, index, flags, q_row=None, s_row=None, q_colT=None, s_colT=None,
                   stream=None):
    p = _address
    check(_functions()["mxfp4_quantize"](p(x), x_rows, rows, cols, ld_x, p(index), flags, p(q_row), p(s_row), p(q_colT),
                                         p(s_colT), _stream(stream)), "mxfp4_quantize")


def mxfp4_dequantize(q, s, rows, cols, out, ld_out, flags, stream=None):
    p = _address
    check(_functions()["mxfp4_dequantize"](p(q), p(s), rows, cols, p(out), ld_out, flags, _stream(stream)),
          "mxfp4_dequantize")


def mxfp4_gemm(a, a_packed, b, b_packed, c, ldc, M, N, K, flags, stream=None):
    p = _address
    check(_functions()["mxfp4_gemm"](p(a), p(a_packed), p(b), p(b_packed), p(c), ldc, M, N, K, flags, _stream(stream)),
          "mxfp4_gemm")


def mxfp4_grouped_gemm(a, a_packed, b, b_packed, offsets, G, c, ldc, M_total, N, K, flags, stream=None):
    p = _address
    check(_functions()["mxfp4_grouped_gemm"](p(a), p(a_packed), p(b), p(b_packed), p(offsets), G, p(c), ldc, M_total, N,
                                             K, flags, _stream(stream)), "mxfp4_grouped_gemm")


# ------------------------------------------------------ allocating helpers

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
    if not isinstance(x, torch.Tensor) or x.dtype is not torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be a BF16 [rows, cols] tensor with unit column stride")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA (HIP) tensor, got %s" % x.device)
    X, C = x.shape
    dev = x.device
    R = X
    if index is not None:
        if colwise:
            raise ValueError("index goes with the rowwise copy alone")
        R = index.numel()
        need(index, "index", torch.int32, (R,), dev)
    flags = (MXFP4_ROWWISE if rowwise else 0) | (MXFP4_COLWISE if colwise else 0) | (MXFP4_PACKED_SCALES if packed else 0)
    out, q, s, qT, sT = {}, None, None, None, None
    if rowwise:
        out["q_row"] = q = torch.empty((R, C // 2), dtype=torch.uint8, device=dev)
        s = (torch.empty((C // 128, R), dtype=torch.int32, device=dev) if packed
             else torch.empty((R, C // 32), dtype=torch.uint8, device=dev))
        out["p_row" if packed else "s_row"] = s
    if colwise:
        out["q_colT"] = qT = torch.empty((C, R // 2), dtype=torch.uint8, device=dev)
        sT = (torch.empty((R // 128, C), dtype=torch.int32, device=dev) if packed
              else torch.empty((C, R // 32), dtype=torch.uint8, device=dev))
        out["p_colT" if packed else "s_colT"] = sT
    launch(_functions()["mxfp4_quantize"], "mxfp4_quantize", dev, x.data_ptr(), X, R, C, max(x.stride(0), C),
           None if index is None else index.data_ptr(), flags, _address(q), _address(s), _address(qT), _address(sT))
    return out


def dequantize(q, scales, out=None, stream=None):
    """BF16 [R, K] values of codes q [R, K / 2] with packed scale words int32
    [K / 128, R] or scale bytes uint8 [R, K / 32]."""
    if stream is not None:
        return on_stream(stream, (q, scales, out), lambda: dequantize(q, scales, out))
    if not isinstance(q, torch.Tensor) or q.dim() != 2 or not isinstance(scales, torch.Tensor):
        raise ValueError("q must be a 2-D tensor of MXFP4 codes, scales a tensor")
    R, half = q.shape
    K = 2 * half
    dev = q.device
    need(q, "q", torch.uint8, (R, half))
    packed = scales.dtype is torch.int32
    if packed:
        need(scales, "scales", torch.int32, (K // 128, R), dev)
    else:
        need(scales, "scales", torch.uint8, (R, K // 32), dev)
    if out is None:
        out = torch.empty((R, K), dtype=torch.bfloat16, device=dev)
    elif out.dtype is not torch.bfloat16 or out.shape != (R, K) or out.stride(1) != 1 or out.device != dev:
        raise ValueError("out must be a BF16 [R, K] tensor with unit column stride on q's device")
    launch(_functions()["mxfp4_dequantize"], "mxfp4_dequantize", dev, q.data_ptr(), scales.data_ptr(), R, K,
           out.data_ptr(), max(out.stride(0), K), MXFP4_PACKED_SCALES if packed else 0)
    return out


def _product(a, a_packed, b, b_packed, b_rows, N, out, accumulate, swiglu):
    """Checks common to both products; returns M, K, the output and the flags."""
    M, half = a.shape
    K = 2 * half
    dev = a.device
    need(a, "a", torch.uint8, (M, half))
    need(a_packed, "a_packed", torch.int32, (K // 128, M), dev)
    need(b_packed, "b_packed", torch.int32, (K // 128, b_rows), dev)
    if accumulate:
        if swiglu:
            raise ValueError("accumulate and swiglu exclude each other")
        if out is None:
            raise ValueError("accumulate=True needs out")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    elif out.dtype is not torch.bfloat16 or out.shape != (M, N) or out.stride(1) != 1 or out.device != dev:
        raise ValueError("out must be a BF16 [M, N] tensor with unit column stride on the operands' device")
    return M, K, out, MXFP4_GEMM_ACCUMULATE if accumulate else MXFP4_GEMM_SWIGLU if swiglu else 0


def gemm(a, a_packed, b, b_packed, out=None, accumulate=False, swiglu=False, stream=None):
    """C = dq(A) dq(B)^T in BF16 for codes a [M, K / 2], b [N, K / 2] and their
    packed scale words.  accumulate=True adds the product to ``out``;
    swiglu=True: b is [2N, K / 2] (gate rows, then up rows) and C [M, N] =
    SiLU(gate product) * up product."""
    if stream is not None:
        return on_stream(stream, (a, a_packed, b, b_packed, out),
                         lambda: gemm(a, a_packed, b, b_packed, out, accumulate, swiglu))
    if not isinstance(a, torch.Tensor) or a.dim() != 2 or not isinstance(b, torch.Tensor) or b.dim() != 2:
        raise ValueError("a and b must be 2-D tensors of MXFP4 codes")
    rows = b.shape[0]
    if swiglu and rows % 2:
        raise ValueError("swiglu=True needs b with an even number of rows (gate rows, then up rows)")
    N = rows // 2 if swiglu else rows
    M, K, c, flags = _product(a, a_packed, b, b_packed, rows, N, out, accumulate, swiglu)
    need(b, "b", torch.uint8, (rows, K // 2), a.device)
    launch(_functions()["mxfp4_gemm"], "mxfp4_gemm", a.device, a.data_ptr(), a_packed.data_ptr(), b.data_ptr(),
           b_packed.data_ptr(), c.data_ptr(), max(c.stride(0), N), M, N, K, flags)
    return c


def grouped_gemm(a, a_packed, b, b_packed, offsets, out=None, accumulate=False, swiglu=False, stream=None):
    """Ragged grouped product: rows offsets[g] .. offsets[g + 1] - 1 of a (int32
    offsets on the device) times expert g of b [G, N, K / 2] (b_packed [K / 128,
    G * N]); swiglu=True: experts of 2N rows, C [M, N].  Rows outside every
    group are not written."""
    if stream is not None:
        return on_stream(stream, (a, a_packed, b, b_packed, offsets, out),
                         lambda: grouped_gemm(a, a_packed, b, b_packed, offsets, out, accumulate, swiglu))
    if not isinstance(a, torch.Tensor) or a.dim() != 2 or not isinstance(b, torch.Tensor) or b.dim() != 3:
        raise ValueError("a must be 2-D [M, K / 2] and b 3-D [G, N, K / 2] tensors of MXFP4 codes")
    G, rows, _ = b.shape
    if swiglu and rows % 2:
        raise ValueError("swiglu=True needs experts with an even number of rows (gate rows, then up rows)")
    N = rows // 2 if swiglu else rows
    M, K, c, flags = _product(a, a_packed, b, b_packed, G * rows, N, out, accumulate, swiglu)
    need(b, "b", torch.uint8, (G, rows, K // 2), a.device)
    need(offsets, "offsets", torch.int32, (G + 1,), a.device)
    launch(_functions()["mxfp4_grouped_gemm"], "mxfp4_grouped_gemm", a.device, a.data_ptr(), a_packed.data_ptr(),
           b.data_ptr(), b_packed.data_ptr(), offsets.data_ptr(), G, c.data_ptr(), max(c.stride(0), N), M, N, K, flags)
    return c
