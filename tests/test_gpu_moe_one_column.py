"""Matrices of one column, whose column stride may be anything."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def test_one_expert():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    log("one expert")
    x = torch.randn((1, 9), device="cuda").t()
    assert x.shape == (9, 1) and x.stride() == (1, 9)
    for scores in ("softmax", "sigmoid"):
        leaf = x.detach().requires_grad_()
        w, ids = moe.route(leaf, 1, scores=scores, renormalize=False)
        want = torch.ones_like(x) if scores == "softmax" else torch.sigmoid(x)
        assert ids.tolist() == [[0]] * 9 and torch.allclose(w, want, rtol=1e-6, atol=0)
        d, = torch.autograd.grad(w, leaf, torch.ones_like(w))
        want = torch.zeros_like(x) if scores == "softmax" else torch.sigmoid(x) * (1 - torch.sigmoid(x))
        assert torch.allclose(d, want, rtol=1e-5, atol=1e-7)


def test_one_hidden_value():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    log("one hidden value")
    y = torch.randn((1, 8), device="cuda").t().requires_grad_()
    position = torch.tensor([[3, 0], [5, -1]], dtype=torch.int32, device="cuda")
    w = torch.randn((2, 2), device="cuda", requires_grad=True)
    out = moe.combine(y, position, w)
    yd, wd = y.detach(), w.detach()
    want = torch.stack((wd[0, 0] * yd[3] + wd[0, 1] * yd[0], wd[1, 0] * yd[5]))
    assert torch.allclose(out, want, rtol=1e-6, atol=1e-6)
    for dout in (torch.randn((2, 1), device="cuda"), torch.randn((1, 2), device="cuda").t(), torch.ones((), device="cuda").expand(2, 1)):
        dy, dw = torch.autograd.grad(out, (y, w), dout, retain_graph=True)
        want = torch.zeros_like(yd)
        want[3], want[0], want[5] = wd[0, 0] * dout[0], wd[0, 1] * dout[0], wd[1, 0] * dout[1]
        assert torch.allclose(dy, want, rtol=1e-6, atol=1e-7)
        want = torch.stack((torch.cat((dout[0] * yd[3], dout[0] * yd[0])), torch.cat((dout[1] * yd[5], torch.zeros(1, device="cuda")))))
        assert torch.allclose(dw, want, rtol=1e-6, atol=1e-7)
