"""A mixture-of-experts layer on the MXFP4 and routing operators, for inference.

    weights, ids = route(x W_router^T)             per token: experts and weights
    plan = dispatch(ids)                           slots sorted by expert
    a = MXFP4(x[plan.token])                       gathered and quantized in one pass
    h = SiLU(a gate^T) * (a up^T)                  grouped product, SwiGLU epilogue
    y = MXFP4(h) down^T                            grouped product
    out[t] = sum_k weights[t, k] y[position[t, k]]

Nothing waits for the GPU: expert boundaries stay on the device, so the layer
can be captured in a graph.
"""

import torch

from . import moe, mxfp4
from ._tensors import no_tangent


class MXFP4MoE(torch.nn.Module):
    """experts of [gate_up: 2 * ffn x hidden, down: hidden x ffn] in MXFP4 (one
    buffer each, quantized by ``load``).  hidden and ffn are multiples of 128.
    scores, groups, top_groups, group_top and renormalize as for ``moe.route``;
    balance=True adds a per-expert choice bias (a buffer).

    router_dtype is the type of the router's weights and of its logits.  BF16, the
    default, rounds a logit by up to 2^-8 of its value, as models trained with a
    BF16 router expect, and experts that lie closer than that may change places.
    torch.float32 multiplies in 32 bits, and ``moe.route`` then orders by the
    logits as they come.  The product is PyTorch's (this library has products of
    block-scaled operands alone), experts / (3 top_k ffn) of the experts' work."""

    def __init__(self, hidden, ffn, experts, top_k, scores="softmax", groups=1, top_groups=1, group_top=2, renormalize=True,
                 balance=False, device=None, router_dtype=torch.bfloat16):
        super().__init__()
        if hidden % 128 or ffn % 128:
            raise ValueError("hidden and ffn must be multiples of 128")
        if router_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("router_dtype must be torch.bfloat16 or torch.float32")
        self.hidden, self.ffn, self.experts, self.top_k = hidden, ffn, experts, top_k
        self.plan = dict(scores=scores, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renormalize)
        u8, i32 = torch.uint8, torch.int32
        self.register_buffer("router", torch.zeros((experts, hidden), dtype=router_dtype, device=device))
        self.register_buffer("bias", torch.zeros(experts, dtype=torch.float32, device=device) if balance else None)
        self.register_buffer("gate_up", torch.zeros((experts, 2 * ffn, hidden // 2), dtype=u8, device=device))
        self.register_buffer("gate_up_scales", torch.zeros((hidden // 128, experts * 2 * ffn), dtype=i32, device=device))
        self.register_buffer("down", torch.zeros((experts, hidden, ffn // 2), dtype=u8, device=device))
        self.register_buffer("down_scales", torch.zeros((ffn // 128, experts * hidden), dtype=i32, device=device))

    @torch.no_grad()
    def load(self, router, gate_up, down, bias=None):
        """Take a router [experts, hidden] and BF16 weights: gate_up [experts,
        2 * ffn, hidden] (gate rows, then up rows), down [experts, hidden, ffn]."""
        self.router.copy_(router)
        if bias is not None:
            self.bias.copy_(bias)
        for codes, scales, w in ((self.gate_up, self.gate_up_scales, gate_up), (self.down, self.down_scales, down)):
            q = mxfp4.quantize(w.reshape(-1, w.shape[-1]).contiguous(), packed=True)
            codes.copy_(q["q_row"].view_as(codes))
            scales.copy_(q["p_row"])
        return self

    @torch.no_grad()
    def forward(self, x):
        """x BF16 [.., hidden] -> BF16 of the same shape, without a gradient (also where x
        requires one)."""
        if x.dtype != torch.bfloat16 or x.shape[-1] != self.hidden:
            raise ValueError("input must be BF16 with %d features" % self.hidden)
        no_tangent("MXFP4MoE", x)
        t = x.reshape(-1, self.hidden).contiguous()
        weights, ids = moe.route(t.to(self.router.dtype) @ self.router.t(), self.top_k, bias=self.bias, **self.plan)
        plan = moe.dispatch(ids, self.experts)
        a = mxfp4.quantize(t, packed=True, index=plan.token)
        h = mxfp4.grouped_gemm(a["q_row"], a["p_row"], self.gate_up, self.gate_up_scales, plan.offsets, swiglu=True)
        a = mxfp4.quantize(h, packed=True)
        y = mxfp4.grouped_gemm(a["q_row"], a["p_row"], self.down, self.down_scales, plan.offsets)
        return moe.combine(y, plan.position, weights).view(x.shape)
