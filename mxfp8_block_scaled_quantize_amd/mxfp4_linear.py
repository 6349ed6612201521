"""MXFP4 linear layer: fprop, dgrad and wgrad on the MXFP4 products.

    fprop   y  = x W^T    A = x rowwise [M][K],           B = W rowwise [N][K]
    dgrad   dx = dy W     A = dy rowwise [M][N],          B = W columnwise copy [K][N]
    wgrad   dW = dy^T x   A = dy columnwise copy [N][M],  B = x columnwise copy [K][M]

As in the MXFP8 layer, columnwise copies are stored transposed, one pass makes
both copies, and only the copies a product reads are made.  Values are rounded
to nearest, gradients included.  x [.., K] and W [N, K] BF16 with tokens, K and N
multiples of 128.

The weight is quantized in every forward pass, from its value of that moment on
the stream of that pass: a copy kept from an earlier call could be stale (a write
through ``.data`` leaves no trace) or not yet written on this stream.  A program
whose weight stays says so with ``freeze_weight``.
"""

import torch

from ._tensors import no_tangent
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


def _alike(old, new):
    return old is not None and new is not None and old.shape == new.shape and old.device == new.device


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


_NO_COPIES = (None, None, None, None)


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
        self._wq, self._wq_of = _NO_COPIES, ()   # frozen copies and (in a tuple) the parameter they are of

    def freeze_weight(self, colwise=False):
        """Quantize the weight now, for all later calls that need no gradient of
        it (colwise=True: the transposed copy too, which the input's gradient
        reads).  Until the next freeze_weight or thaw_weight the layer does not
        look at the parameter; loading a state dict, moving the module and
        replacing the parameter end it too.  Copies of the same shape are written in
        place, so a graph captured with them follows.  Waits for the device before
        and after, so that they can be used on any stream; not during a capture."""
        w = self.weight.detach()
        if w.is_cuda and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("freeze_weight cannot run while a graph is captured")
        # usable in a later backward pass even if this is called in inference mode
        with torch.inference_mode(False), torch.no_grad():
            old = self._wq if self._is_frozen() else _NO_COPIES
            fresh = _copies(w.contiguous(), True, colwise or old[2] is not None)
            self._wait(w)
            self._wq = tuple(o.copy_(t) if _alike(o, t) else t for o, t in zip(old, fresh))
            self._wq_of = (self.weight,)
            self._wait(w)
        return self

    def thaw_weight(self):
        """Give up the copies of freeze_weight, once the device is done with them."""
        if self._wq[0] is not None:
            self._wait(self._wq[0])
        self._wq, self._wq_of = _NO_COPIES, ()
        return self

    @staticmethod
    def _wait(t):
        if t.is_cuda:
            torch.cuda.synchronize(t.device)

    def _is_frozen(self):
        return bool(self._wq_of) and self._wq_of[0] is self.weight

    def _apply(self, *args, **kwargs):
        self.thaw_weight()
        return super()._apply(*args, **kwargs)

    def _load_from_state_dict(self, *args, **kwargs):
        self.thaw_weight()
        return super()._load_from_state_dict(*args, **kwargs)

    def quantized_weight(self, colwise=True):
        """(q_row, p_row, q_colT, p_colT): the frozen copies, or those of the
        parameter's present value (the transposed one None without colwise)."""
        if self._is_frozen() and not (colwise and self._wq[2] is None):
            return self._wq
        with torch.no_grad():
            return _copies(self.weight.detach().contiguous(), True, colwise)

    def forward(self, x):
        no_tangent("MXFP4Linear", x, self.weight)
        if torch.is_grad_enabled() and (x.requires_grad or self.weight.requires_grad):
            # a weight in training is quantized there, a frozen one may be kept
            frozen = self.quantized_weight(x.requires_grad) if not self.weight.requires_grad else None
            return MXFP4LinearFunction.apply(x, self.weight, frozen)
        if x.dtype != torch.bfloat16 or x.shape[-1] != self.in_features:
            raise ValueError("input must be BF16 with %d features" % self.in_features)
        q = quantize(x.reshape(-1, x.shape[-1]).contiguous(), packed=True)
        w = self.quantized_weight(colwise=False)
        return gemm(q["q_row"], q["p_row"], w[0], w[1]).view(*x.shape[:-1], self.out_features)
