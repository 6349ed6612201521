"""The MXFP4 linear layer and the mixture-of-experts layer."""

import numpy as np
import pytest

import mx4_util as ref
from gpu_util import bf16_to_f64, need_gpu, to_host

pytestmark = pytest.mark.gpu


def _values(t):
    """64-bit values of the MXFP4 copy of t [R, C] along its last axis."""
    codes, scales = ref.quantize(to_host(t.contiguous()))
    return ref.dequantize(codes, scales)


def _near(got, x, y, label):
    """got = bf16(x y^T) for 64-bit operands: fp32 sums of K terms, one rounding."""
    want, err = x @ y.T, x.shape[1] * 2.0 ** -24 * (np.abs(x) @ np.abs(y).T)
    assert np.all(np.abs(bf16_to_f64(to_host(got)) - want) <= err + 2.0 ** -8 * (np.abs(want) + err)), label


def test_linear_forward_and_gradients():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd.mxfp4_linear import MXFP4Linear
    layer = MXFP4Linear(256, 384, device="cuda")
    x = torch.randn((2, 128, 256), device="cuda").bfloat16().requires_grad_()
    dy = torch.randn((2, 128, 384), device="cuda").bfloat16()
    y = layer(x)
    y.backward(dy)
    x2, d2, w = x.detach().view(-1, 256), dy.view(-1, 384), layer.weight.detach()
    _near(y.detach().view(-1, 384), _values(x2), _values(w), "y")
    _near(x.grad.view(-1, 256), _values(d2), _values(w.t()), "dx")
    _near(layer.weight.grad, _values(d2.t()), _values(x2.t()), "dw")


def test_linear_makes_only_what_is_needed_and_follows_the_weight():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd.mxfp4_linear import MXFP4Linear, MXFP4LinearFunction
    layer = MXFP4Linear(128, 256, device="cuda")
    x = torch.randn((5, 128), device="cuda").bfloat16()
    with torch.no_grad():
        y = layer(x)                                    # any number of tokens
    _near(y, _values(x), _values(layer.weight.detach()), "inference")
    assert layer._wq[2] is None
    with torch.no_grad():
        layer.weight.mul_(-2.0)
        _near(layer(x), _values(x), _values(layer.weight.detach()), "after an update")
    x = torch.randn((128, 128), device="cuda").bfloat16()
    dy = torch.randn((128, 256), device="cuda").bfloat16()
    w = layer.weight.detach()
    xg, wg = x.clone().requires_grad_(), w.clone().requires_grad_()
    MXFP4LinearFunction.apply(xg, w).backward(dy)
    MXFP4LinearFunction.apply(x, wg).backward(dy)
    _near(xg.grad, _values(dy), _values(w.t()), "dx alone")
    _near(wg.grad, _values(dy.t()), _values(x.t()), "dw alone")
    with pytest.raises(ValueError, match="multiples of 128"):
        layer(torch.randn((100, 128), device="cuda").bfloat16().requires_grad_())
    with pytest.raises(TypeError, match="BF16"):
        MXFP4LinearFunction.apply(x.float(), w)


@pytest.mark.parametrize("tokens", [1, 3, 50, 700])
@pytest.mark.parametrize("kw", [dict(), dict(scores="sigmoid", groups=4, top_groups=2, balance=True)], ids=["softmax", "grouped"])
def test_moe_layer(tokens, kw):
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd.moe_layer import MXFP4MoE
    H, F, E, K = 256, 384, 16, 4
    g = torch.Generator(device="cuda").manual_seed(tokens)
    layer = MXFP4MoE(H, F, E, K, device="cuda", **kw)
    router = torch.randn((E, H), generator=g, device="cuda").bfloat16() * 0.2
    gate_up = torch.randn((E, 2 * F, H), generator=g, device="cuda").bfloat16() * 0.1
    down = torch.randn((E, H, F), generator=g, device="cuda").bfloat16() * 0.1
    bias = torch.randn(E, generator=g, device="cuda") * 0.05 if kw.get("balance") else None
    layer.load(router, gate_up, down, bias)
    x = torch.randn((tokens, H), generator=g, device="cuda").bfloat16()
    out = bf16_to_f64(to_host(layer(x)))
    # the layer in 64 bits, each product's result rounded to BF16 as the layer stores it
    logits = bf16_to_f64(to_host(x @ router.t()))
    plan = {k: v for k, v in kw.items() if k != "balance"}
    w, ids, _ = ref.route(logits, K, plan.pop("scores", "softmax"), bias=None if bias is None else bias.cpu().numpy(), **plan)
    vx, vu, vd = _values(x), _values(gate_up.view(-1, H)).reshape(E, 2 * F, H), _values(down.view(-1, F)).reshape(E, H, F)
    want, size = np.zeros((tokens, H)), np.zeros((tokens, H))
    for t in range(tokens):
        for k in range(K):
            e = ids[t, k]
            gate, up = vu[e][:F] @ vx[t], vu[e][F:] @ vx[t]
            h = torch.from_numpy(gate / (1 + np.exp(-gate)) * up).bfloat16()
            y = vd[e] @ _values(h[None])[0]
            want[t] += w[t, k] * y
            size[t] += w[t, k] * (np.abs(vd[e]) @ np.abs(_values(h[None])[0]))
    # an h next to a rounding border may take the other BF16 value and then the
    # other E2M1 code, half an E2M1 step (at most 1/4 of the value) of one term
    # in the sum: far below 2% of the terms' sizes; y and out are rounded to BF16
    assert np.all(np.abs(out - want) <= 0.02 * size + 2.0 ** -7 * np.abs(want))
    assert np.mean(np.abs(out - want) <= 2.0 ** -7 * size) > 0.99


def test_moe_layer_refusals():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd.moe_layer import MXFP4MoE
    with pytest.raises(ValueError, match="multiples of 128"):
        MXFP4MoE(200, 128, 4, 2)
    layer = MXFP4MoE(128, 128, 4, 2, device="cuda")
    with pytest.raises(ValueError, match="BF16 with 128"):
        layer(torch.zeros((2, 256), dtype=torch.bfloat16, device="cuda"))
