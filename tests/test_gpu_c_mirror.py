"""The functions that mirror the C ABI of include/mxfp4.h and include/moe.h, on
tensors of the caller's own: the same results as the allocating helpers."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def _empty(torch, like):
    return torch.full_like(like, 77)


@pytest.mark.parametrize("side", [False, True])
def test_mxfp4(side):
    torch = need_gpu()
    import mxfp8_block_scaled_quantize_amd as mx
    from mxfp8_block_scaled_quantize_amd import mxfp4
    log("C mirror of MXFP4, side stream %s" % side)
    R, C, N = 128, 256, 64
    x = torch.randn((R, C + 8), device="cuda").bfloat16()[:, :C]
    want = mxfp4.quantize(x, rowwise=True, colwise=True, packed=True)
    b = mxfp4.quantize(torch.randn((N, C), device="cuda").bfloat16(), packed=True)
    index = torch.tensor([3, -1, 5], dtype=torch.int32, device="cuda")
    gathered = mxfp4.quantize(x, packed=True, index=index)
    offsets = torch.tensor([0, 50, R], dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    if side:
        stream.wait_stream(torch.cuda.current_stream())
    got = {k: _empty(torch, v) for k, v in want.items()}
    few = {k: _empty(torch, v) for k, v in gathered.items()}
    values, c, grouped = (torch.full(s, 7.0, dtype=torch.bfloat16, device="cuda") for s in ((R, C), (R, N), (R, N // 2)))
    torch.cuda.synchronize()
    both = mxfp4.MXFP4_ROWWISE | mxfp4.MXFP4_COLWISE | mxfp4.MXFP4_PACKED_SCALES
    mxfp4.mxfp4_quantize(x, R, R, C, x.stride(0), None, both, got["q_row"], got["p_row"], got["q_colT"], got["p_colT"],
                         stream=stream)
    mxfp4.mxfp4_quantize(x, R, 3, C, x.stride(0), index, mxfp4.MXFP4_ROWWISE | mxfp4.MXFP4_PACKED_SCALES, few["q_row"],
                         few["p_row"], stream=stream)
    mxfp4.mxfp4_dequantize(got["q_row"], got["p_row"], R, C, values, C, mxfp4.MXFP4_PACKED_SCALES, stream=stream)
    mxfp4.mxfp4_gemm(got["q_row"], got["p_row"], b["q_row"], b["p_row"], c, N, R, N, C, 0,
                     stream=stream.cuda_stream if side else None)
    mxfp4.mxfp4_grouped_gemm(got["q_row"], got["p_row"], b["q_row"], b["p_row"], offsets, 2, grouped, N // 2, R, N // 2, C, 0,
                             stream=stream)
    torch.cuda.synchronize()
    for have, wanted in ((got, want), (few, gathered)):
        assert all(torch.equal(have[k], v) for k, v in wanted.items())
    assert torch.equal(values, mxfp4.dequantize(want["q_row"], want["p_row"]))
    assert torch.equal(c, mxfp4.gemm(want["q_row"], want["p_row"], b["q_row"], b["p_row"]))
    assert torch.equal(grouped, mxfp4.grouped_gemm(want["q_row"], want["p_row"], b["q_row"].view(2, N // 2, C // 2),
                                                   b["p_row"], offsets))
    with pytest.raises(mx.MXFP8Error, match="mxfp4_gemm"):
        mxfp4.mxfp4_gemm(got["q_row"], got["p_row"], b["q_row"], b["p_row"], c, N, R, N, C + 1, 0)


@pytest.mark.parametrize("side", [False, True])
def test_moe(side):
    torch = need_gpu()
    import mxfp8_block_scaled_quantize_amd as mx
    from mxfp8_block_scaled_quantize_amd import moe
    log("C mirror of MoE, side stream %s" % side)
    T, E, K, H = 5000, 32, 4, 64          # enough slots for a dispatch with a workspace
    logits = torch.randn((T, E), device="cuda").requires_grad_()
    bias = torch.randn(E, device="cuda") * 0.05
    w, ids = moe.route(logits, K, bias=bias, groups=4, top_groups=2)
    dw = torch.randn((T, K), device="cuda")
    dlogits, = torch.autograd.grad(w, logits, dw)
    w, logits = w.detach(), logits.detach()
    plan = moe.dispatch(ids, E)
    y = torch.randn((T * K, H), device="cuda").bfloat16().requires_grad_()
    leaf = w.clone().requires_grad_()
    out = moe.combine(y, plan.position, leaf)
    dout = torch.randn((T, H), device="cuda").bfloat16()
    dy, dweights = torch.autograd.grad(out, (y, leaf), dout)
    y, out = y.detach(), out.detach()
    stream = torch.cuda.Stream() if side else None
    bytes_ = moe.moe_dispatch_workspace_bytes(T, E, K)
    assert bytes_ > 0
    work = torch.empty(max(bytes_, 4 * T * K), dtype=torch.uint8, device="cuda")
    got = [_empty(torch, t) for t in (w, ids, dlogits, *plan, out, dy, dweights)]
    gw, gi, gd, go, gt, gp, gout, gdy, gdw = got
    torch.cuda.synchronize()
    flags = moe.MOE_ROUTE_RENORMALIZE
    moe.moe_route(logits, moe.MOE_FP32, T, E, E, bias, K, 4, 2, 2, flags, gw, gi, stream=stream)
    moe.moe_route_backward(logits, moe.MOE_FP32, T, E, E, gi, dw, K, flags, gd, stream=stream)
    moe.moe_dispatch(gi, T, E, K, go, gt, gp, work, work.numel(), stream=stream)
    moe.moe_combine(y, moe.MOE_BF16, T * K, H, gp, gw, T, K, H, gout, stream=stream.cuda_stream if side else None)
    moe.moe_combine_backward(y, moe.MOE_BF16, T * K, H, gp, gw, T, K, H, dout, H, gdy, gdw, work, work.numel(), stream=stream)
    torch.cuda.synchronize()
    for have, want in zip(got, (w, ids, dlogits, *plan, out, dy, dweights)):
        assert torch.equal(have, want)
    with pytest.raises(mx.MXFP8Error, match="moe_dispatch"):
        moe.moe_dispatch(gi, T, E, K, go, gt, gp, None, 0)
