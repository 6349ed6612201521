"""An attention layer on the paged MXFP4 cache, for inference.

    q, k, v = MXFP4(x) W_qkv^T                      one product
    q, k = rotate(q, k)                             by the positions of the rows
    cache[slots] = MXFP4(k), MXFP4(v)
    a = softmax(scale q k^T) v                      over each request's pages
    out = MXFP4(a) W_out^T

Lengths, tables, slots and positions stay on the device, so a step of it can be
captured in a graph.
"""

import torch

from . import kvcache, mxfp4, rotary
from ._tensors import no_tangent


class MXFP4Attention(torch.nn.Module):
    """heads queries and kv_heads keys and values of head_dim, projected from and to
    ``hidden`` features with weights in MXFP4 (``load``).  hidden and heads * head_dim
    are multiples of 128.  turns and magnitude: the frequencies of ``rotary.turns`` (None:
    no rotary positions; 64 bits, also after a cast of the module); interleaved, window and
    scale as for ``rotary.rotate`` and ``kvcache.attention``."""

    def __init__(self, hidden, heads, kv_heads, head_dim, turns=None, magnitude=1.0, interleaved=False, window=0, scale=None,
                 device=None):
        super().__init__()
        if hidden % 128 or heads * head_dim % 128:
            raise ValueError("hidden and heads * head_dim must be multiples of 128")
        if head_dim not in (64, 128, 256):
            raise ValueError("head_dim must be 64, 128 or 256")
        if kv_heads < 1 or heads < 1 or heads % kv_heads:
            raise ValueError("kv_heads must divide heads")
        self.hidden, self.heads, self.kv_heads, self.head_dim = hidden, heads, kv_heads, head_dim
        self.magnitude, self.interleaved, self.window, self.scale = magnitude, interleaved, window, scale
        rows, width = (heads + 2 * kv_heads) * head_dim, heads * head_dim
        u8, i32 = torch.uint8, torch.int32
        self.register_buffer("turns", None if turns is None else turns.to(device=device, dtype=torch.float64))
        self.register_buffer("qkv", torch.zeros((rows, hidden // 2), dtype=u8, device=device))
        self.register_buffer("qkv_scales", torch.zeros((hidden // 128, rows), dtype=i32, device=device))
        self.register_buffer("out", torch.zeros((hidden, width // 2), dtype=u8, device=device))
        self.register_buffer("out_scales", torch.zeros((width // 128, hidden), dtype=i32, device=device))

    def _apply(self, fn, recurse=True):
        # a cast of the module (``.to(torch.bfloat16)``, ``.half()``) moves the frequencies and leaves their 64 bits
        turns = self.turns
        super()._apply(fn, recurse)
        if turns is not None and self.turns.dtype != turns.dtype:
            self.turns = turns.to(self.turns.device)
        return self

    @torch.no_grad()
    def load(self, qkv, out):
        """Take BF16 weights: qkv [(heads + 2 kv_heads) * head_dim, hidden] (rows of the
        queries, the keys, the values), out [hidden, heads * head_dim]."""
        for codes, scales, w in ((self.qkv, self.qkv_scales, qkv), (self.out, self.out_scales, out)):
            q = mxfp4.quantize(w.contiguous(), packed=True)
            codes.copy_(q["q_row"].view_as(codes))
            scales.copy_(q["p_row"])
        return self

    def forward(self, x, cache, table, plan, max_queries=None):
        """x BF16 [tokens, hidden], the rows that ``kvcache.extend`` planned (plan, with
        the cache's table) -> BF16 of the same shape; the rows' keys and values are
        written to the cache.  What a row that belongs to no request comes out as means
        nothing, nor do the rows of a request that got no slots.  max_queries, the longest
        run of new tokens of a request, as for ``kvcache.attention``: without it a step of
        single tokens takes the kernel for prompts.  There is no gradient: an x that requires one is refused
        while gradients are enabled."""
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != self.hidden:
            raise ValueError("input must be a BF16 [tokens, %d] tensor" % self.hidden)
        if x.requires_grad and torch.is_grad_enabled():
            raise ValueError("input requires a gradient, which MXFP4Attention does not have: call it with gradients disabled")
        no_tangent("MXFP4Attention", x)
        with torch.no_grad():
            return self._step(x, cache, table, plan, max_queries)

    def _step(self, x, cache, table, plan, max_queries):
        h, hkv = self.heads, self.kv_heads
        a = mxfp4.quantize(x.contiguous(), packed=True)
        q, k, v = mxfp4.gemm(a["q_row"], a["p_row"], self.qkv, self.qkv_scales).view(
            x.shape[0], h + 2 * hkv, self.head_dim).split((h, hkv, hkv), 1)
        if self.turns is not None:
            q, k = rotary.rotate(q, k, plan.positions, self.turns, interleaved=self.interleaved, magnitude=self.magnitude)
        kvcache.append(cache, k, v, plan.slots)
        y = kvcache.attention(q, cache, table, plan.lengths, plan.offsets, scale=self.scale, window=self.window,
                              max_queries=max_queries)
        a = mxfp4.quantize(y.view(x.shape[0], h * self.head_dim), packed=True)
        return mxfp4.gemm(a["q_row"], a["p_row"], self.out, self.out_scales)
