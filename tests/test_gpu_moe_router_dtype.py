"""The mixture-of-experts layer's router in 32 bits."""

import pytest
import torch

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def test_logits_closer_than_bf16():
    need_gpu()
    from mxfp8_block_scaled_quantize_amd.moe_layer import MXFP4MoE
    log("router dtype")
    H, F, E, K, T = 128, 128, 16, 2, 5
    g = torch.Generator(device="cuda").manual_seed(0)
    gate_up = (torch.randn((E, 2 * F, H), generator=g, device="cuda") * 0.1).bfloat16()
    down = (torch.randn((E, H, F), generator=g, device="cuda") * 0.1).bfloat16()
    # logits 1 + e 2^-12 of x's first feature: all 1 in BF16
    router = torch.zeros((E, H), device="cuda")
    router[:, 0] = 1 + torch.arange(E, device="cuda") * 2.0 ** -12
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    x[:, 0] = 1
    out = {}
    for dtype in (torch.bfloat16, torch.float32):
        layer = MXFP4MoE(H, F, E, K, device="cuda", router_dtype=dtype).load(router, gate_up, down)
        assert layer.router.dtype == dtype
        out[dtype] = layer(x)
    # the same experts, put where the choice falls on them
    last = MXFP4MoE(H, F, E, K, device="cuda").load(torch.flip(router, (0,)), torch.flip(gate_up, (0,)), torch.flip(down, (0,)))
    assert torch.equal(MXFP4MoE(H, F, E, K, device="cuda").load(router, gate_up, down)(x), out[torch.bfloat16])
    close = (out[torch.float32].double() - last(x).double()).abs()
    assert torch.all(close <= 2.0 ** -6 * last(x).double().abs() + 2.0 ** -9)   # weights 0.5 either way, to 2^-12
    assert (out[torch.float32].double() - out[torch.bfloat16].double()).abs().max() > 0.05
    with pytest.raises(ValueError, match="router_dtype"):
        MXFP4MoE(H, F, E, K, router_dtype=torch.float16)
