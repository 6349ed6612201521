"""MXFP4 linear layer: fprop, dgrad and wgrad on the MXFP4 products.

    fprop   y  = x W^T    A = x rowwise [M][K],           B = W rowwise [N][K]
    dgrad   dx = dy W     A = dy rowwise [M][N],          B = W columnwise copy [K][N]
    wgrad   dW = dy^T x   A = dy columnwise copy [N][M],  B = x columnwise copy [K][M]

As in the MXFP8 layer, columnwise copies are stored transposed, one pass makes
both copies, only the copies a product reads are made, and the weight's copies
are kept until the parameter changes.  Values are rounded to nearest, gradients
included.  x [.., K] and W [N, K] BF16 with tokens, K and N multiples of 128.
"""

import torch

from .mxfp4 import gemm, quantize


def _copies(t, row, col):
    """(q_row, p_row, q_colT, p_colT) of t, None for a copy that is not asked for."""
    q = quantize(t, rowwise=row, colwise=col, packed=True)
    return q.get("q_row"), q.get("p_row"), q.get("q_colT"), q.get("p_colT")


def _matrix(x, weight):
    if x.dtype != torch.bfloat16 or weight.dtype != torch.bfloat16:
        raise TypeError("MXFP4 linear takes BF16 input and weight")
    x2 = x.reshape(-1, x.shape[-1]).contiguous()
    M, K = x2.shape
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError("weight is [%d, %d], input has %d features" % (weight.shape[0], weight.shape[1], K))
    if M % 128 or N % 128 or K % 128:
        raise ValueError("MXFP4 linear needs tokens, in- and out-features to be multiples of 128 "
                         "(got M=%d, K=%d, N=%d)" % (M, K, N))
    return x2


class MXFP4LinearFunction(torch.autograd.Function):
    """apply(x, weight, weight_q=None): weight_q, when given, is the weight's
    quantization (q_row, p_row, q_colT, p_colT) from its current value."""

    @staticmethod
    def forward(ctx, x, weight, weight_q=None):
        x2 = _matrix(x, weight)
        want_dx, want_dw = ctx.needs_input_grad[:2]
        qx, px, qxT, pxT = _copies(x2, True, want_dw)
        if weight_q is None:
            weight_q = _copies(weight.contiguous(), True, want_dx)
        qw, pw, qwT, pwT = weight_q
        ctx.save_for_backward(qxT, pxT, *((qwT, pwT) if want_dx else (None, None)))
        ctx.shape = x.shape
        return gemm(qx, px, qw, pw).view(*x.shape[:-1], weight.shape[0])

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        qxT, pxT, qwT, pwT = ctx.saved_tensors
        want_dx, want_dw = ctx.needs_input_grad[:2]
        if not (want_dx or want_dw):
            return None, None, None
        dy2 = dy.reshape(-1, dy.shape[-1]).to(torch.bfloat16).contiguous()
        qd, pd, qdT, pdT = _copies(dy2, want_dx, want_dw)
        dx = gemm(qd, pd, qwT, pwT).view(ctx.shape) if want_dx else None
        dw = gemm(qdT, pdT, qxT, pxT) if want_dw else None
        return dx, dw, None


class MXFP4Linear(torch.nn.Module):
    """y = x W^T with MXFP4 fprop, dgrad and wgrad.  Without a gradient to come
    any number of tokens is allowed (no copy is reduced over them)."""

    def __init__(self, in_features, out_features, device=None):
        super().__init__()
        if in_features % 128 or out_features % 128:
            raise ValueError("in- and out-features must be multiples of 128")
        self.in_features, self.out_features = in_features, out_features
        w = torch.empty((out_features, in_features), dtype=torch.bfloat16, device=device)
        torch.nn.init.normal_(w, std=in_features ** -0.5)
        self.weight = torch.nn.Parameter(w)
        self._wq_key = None
        self._wq = None

    def quantized_weight(self, colwise=True):
        """The weight's copies, made again only when the parameter's storage,
        shape or version counter has changed (or the transposed one is wanted
        for the first time)."""
        w = self.weight
        key = (w.data_ptr(), w.device, tuple(w.shape), w._version)
        if self._wq is None or self._wq_key != key or (colwise and self._wq[2] is None):
            with torch.no_grad():
                self._wq = _copies(w.detach().contiguous(), True, colwise)
            self._wq_key = key
        return self._wq

    def forward(self, x):
        if torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad):
            return MXFP4LinearFunction.apply(x, self.weight, self.quantized_weight())
        if x.dtype != torch.bfloat16 or x.shape[-1] != self.in_features:
            raise ValueError("input must be BF16 with %d features" % self.in_features)
        q = quantize(x.reshape(-1, x.shape[-1]).contiguous(), packed=True)
        w = self.quantized_weight(colwise=False)
        return gemm(q["q_row"], q["p_row"], w[0], w[1]).view(*x.shape[:-1], self.out_features)
