"""MXFP8 products written into a caller's tensor (out=) move its version."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def _calls(torch):
    import mxfp8_block_scaled_quantize_amd as mx
    g = torch.Generator(device="cuda").manual_seed(1)
    qa = mx.quantize(torch.randn((64, 256), generator=g, device="cuda").bfloat16(), packed=True)
    qb = mx.quantize(torch.randn((128, 256), generator=g, device="cuda").bfloat16(), packed=True)
    a, ap, b, bp = qa["q_row"], qa["p_row"], qb["q_row"], qb["p_row"]
    offsets = torch.tensor([0, 30, 64], dtype=torch.int32, device="cuda")
    return {
        "gemm": ((64, 128), lambda out: mx.gemm(a, ap, b, bp, out=out)),
        "accumulate": ((64, 128), lambda out: mx.gemm(a, ap, b, bp, out=out, accumulate=True)),
        "bias": ((64, 128), lambda out: mx.gemm(a, ap, b, bp, out=out, bias=torch.zeros(128, dtype=torch.bfloat16, device="cuda"))),
        "grouped": ((64, 64), lambda out: mx.grouped_gemm(a, ap, b.view(2, 64, 256), bp, offsets, out=out)),
    }


@pytest.mark.parametrize("name", ["gemm", "accumulate", "bias", "grouped"])
def test_saved_tensor_overwritten(name):
    torch = need_gpu()
    shape, call = _calls(torch)[name]
    log("MXFP8 saved tensor overwritten by %s" % name)
    saved = torch.ones(shape, dtype=torch.bfloat16, device="cuda")
    leaf = torch.ones(shape, dtype=torch.bfloat16, device="cuda", requires_grad=True)
    y = leaf * saved
    before = saved._version
    assert call(saved) is saved and saved._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        call(torch.zeros(shape, dtype=torch.bfloat16, device="cuda"))


def test_layer_sees_a_weight_written_through_out():
    torch = need_gpu()
    import mxfp8_block_scaled_quantize_amd as mx
    from mxfp8_block_scaled_quantize_amd.linear import MXFP8Linear
    log("MXFP8 layer weight through out")
    layer, other = MXFP8Linear(128, 256, device="cuda"), MXFP8Linear(128, 256, device="cuda")
    x = torch.randn((128, 128), device="cuda").bfloat16()
    qa = mx.quantize(torch.randn((256, 128), device="cuda").bfloat16(), packed=True)
    qb = mx.quantize(torch.randn((128, 128), device="cuda").bfloat16(), packed=True)
    with torch.no_grad():
        layer(x)
        mx.gemm(qa["q_row"], qa["p_row"], qb["q_row"], qb["p_row"], out=layer.weight)
        other.weight.copy_(layer.weight)
        assert torch.equal(layer(x), other(x))
