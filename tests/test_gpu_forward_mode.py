"""Forward-mode derivatives: the operators and layers have none, and say so
instead of dropping a tangent."""

import pytest
import torch
import torch.autograd.forward_ad as fwad

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def _dual(t):
    return fwad.make_dual(t, torch.ones_like(t))


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", ["logits", "bias"])
def test_route(which, grad):
    need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    log("forward mode: route %s grad=%s" % (which, grad))
    logits, bias = torch.randn((4, 16), device="cuda", requires_grad=grad), torch.zeros(16, device="cuda")
    with fwad.dual_level():
        moe.route(logits, 2, bias=bias)
        args = (_dual(logits), bias) if which == "logits" else (logits, _dual(bias))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            moe.route(args[0], 2, bias=args[1])
    moe.route(logits, 2, bias=bias)


@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("which", ["y", "weights"])
def test_combine(which, grad):
    need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    log("forward mode: combine %s grad=%s" % (which, grad))
    y, w = torch.randn((8, 32), device="cuda", requires_grad=grad), torch.randn((4, 2), device="cuda")
    position = torch.arange(8, device="cuda", dtype=torch.int32).view(4, 2)
    with fwad.dual_level():
        moe.combine(y, position, w)
        args = (_dual(y), w) if which == "y" else (y, _dual(w))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            moe.combine(args[0], position, args[1])
        with pytest.raises(NotImplementedError, match="forward-mode"), torch.no_grad():
            moe.combine(args[0], position, args[1])


def test_out():
    need_gpu()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    log("forward mode: out")
    x = torch.randn((32, 128), device="cuda").bfloat16()
    q = mxfp4.quantize(x, packed=True)
    with fwad.dual_level():
        with pytest.raises(NotImplementedError, match="forward-mode"):
            mxfp4.dequantize(q["q_row"], q["p_row"], out=_dual(x))
        with pytest.raises(NotImplementedError, match="forward-mode"):
            mxfp4.gemm(q["q_row"], q["p_row"], q["q_row"], q["p_row"], out=_dual(torch.zeros((32, 32), device="cuda").bfloat16()))


@pytest.mark.parametrize("which", ["input", "weight"])
@pytest.mark.parametrize("frozen", [False, True])
def test_layers(frozen, which):
    need_gpu()
    from mxfp8_block_scaled_quantize_amd.linear import MXFP8Linear
    from mxfp8_block_scaled_quantize_amd.moe_layer import MXFP4MoE
    from mxfp8_block_scaled_quantize_amd.mxfp4_linear import MXFP4Linear
    log("forward mode: layers frozen=%s" % frozen)
    x = torch.randn((128, 128), device="cuda").bfloat16()
    layers = [MXFP4Linear(128, 128, device="cuda"), MXFP8Linear(128, 128, device="cuda", bias=True)]
    if which == "input":
        layers.append(MXFP4MoE(128, 128, 4, 2, device="cuda"))
    for layer in layers:
        if frozen and hasattr(layer, "weight"):
            layer.requires_grad_(False)
        with fwad.dual_level():
            layer(x)
            if which == "weight":
                del layer.weight
                layer.weight = _dual(torch.randn((128, 128), device="cuda").bfloat16())
                dual = x
            else:
                dual = _dual(x)
            with pytest.raises(NotImplementedError, match="forward-mode"):
                layer(dual)
            with pytest.raises(NotImplementedError, match="forward-mode"), torch.no_grad():
                layer(dual)
        if which == "input":
            layer(x)
