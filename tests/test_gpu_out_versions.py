"""Tensors that a call writes into (out=) count as written: their version moves,
so that autograd notices, and one that requires a gradient is refused."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu

N, K = 128, 256


def _operand(torch, rows, seed):
    from mxfp8_block_scaled_quantize_amd import mxfp4
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = mxfp4.quantize(torch.randn((rows, K), generator=g, device="cuda").bfloat16(), packed=True)
    return q["q_row"], q["p_row"]


def _calls(torch):
    """Name -> (shape of out, call with out)."""
    from mxfp8_block_scaled_quantize_amd import mxfp4
    a, ap = _operand(torch, 64, 1)
    b, bp = _operand(torch, N, 2)
    offsets = torch.tensor([0, 40, 64], dtype=torch.int32, device="cuda")
    experts = b.view(2, N // 2, K // 2)
    return {
        "dequantize": ((64, K), lambda out: mxfp4.dequantize(a, ap, out=out)),
        "gemm": ((64, N), lambda out: mxfp4.gemm(a, ap, b, bp, out=out)),
        "accumulate": ((64, N), lambda out: mxfp4.gemm(a, ap, b, bp, out=out, accumulate=True)),
        "swiglu": ((64, N // 2), lambda out: mxfp4.gemm(a, ap, b, bp, out=out, swiglu=True)),
        "grouped": ((64, N // 2), lambda out: mxfp4.grouped_gemm(a, ap, experts, bp, offsets, out=out)),
    }


NAMES = ["dequantize", "gemm", "accumulate", "swiglu", "grouped"]


@pytest.mark.parametrize("name", NAMES)
def test_version_moves(name):
    torch = need_gpu()
    shape, call = _calls(torch)[name]
    log("out version of %s" % name)
    out = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    before = out._version
    assert call(out).data_ptr() == out.data_ptr()
    assert out._version > before
    # a view's version is its base's
    base = torch.zeros((shape[0] + 1, shape[1] + 64), dtype=torch.bfloat16, device="cuda")
    before = base._version
    call(base[1:, 64:])
    assert base._version > before
    with torch.inference_mode():       # such tensors have no version
        call(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))


@pytest.mark.parametrize("name", NAMES)
def test_saved_tensor_overwritten(name):
    torch = need_gpu()
    shape, call = _calls(torch)[name]
    log("saved tensor overwritten by %s" % name)
    saved = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    leaf = torch.ones(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = leaf * saved
    call(saved)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


@pytest.mark.parametrize("name", NAMES)
def test_out_that_requires_a_gradient(name):
    torch = need_gpu()
    shape, call = _calls(torch)[name]
    log("out with a gradient: %s" % name)
    leaf = torch.ones(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    for out in (leaf, leaf * 1):
        with pytest.raises(ValueError, match="out requires a gradient"):
            call(out)
    assert torch.equal(leaf.detach(), torch.ones_like(leaf))
    with torch.no_grad():              # writing a parameter's value
        before = leaf._version
        call(leaf)
        assert leaf._version > before and leaf.requires_grad and leaf.is_leaf


def test_layer_sees_a_weight_written_through_out():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    from mxfp8_block_scaled_quantize_amd.mxfp4_linear import MXFP4Linear
    layer = MXFP4Linear(K, N, device="cuda")
    x = torch.randn((7, K), device="cuda").bfloat16()
    q, p = _operand(torch, N, 5)
    with torch.no_grad():
        layer(x)
        mxfp4.dequantize(q, p, out=layer.weight)
        got = layer(x)
        other = MXFP4Linear(K, N, device="cuda")
        other.weight.copy_(mxfp4.dequantize(q, p))
        assert torch.equal(got, other(x))
