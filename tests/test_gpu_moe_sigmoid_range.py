"""Sigmoid routing where exp(-logit) leaves fp32's range: finite logits from -87
to -105, whose scores are 1e-38 and less, against 64 bits."""

import numpy as np
import pytest

import mx4_util as ref
from gpu_util import log, need_gpu, to_host

pytestmark = pytest.mark.gpu

FLUSH = 2.0 ** -126   # scores below fp32's normal range may count as 0


def _moe():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    return torch, moe


def _far_logits(torch, T, E, dtype, seed):
    """Three experts in 32 with ordinary logits, the others far below."""
    g = torch.Generator().manual_seed(seed)
    far = torch.rand((T, E), generator=g) * 18 - 105
    near = torch.randn((T, E), generator=g)
    return torch.where(torch.rand((T, E), generator=g) < 3 / 32, near, far).to(getattr(torch, dtype))


# tokens, experts, top_k, bias, groups, top_groups, group_top
SHAPES = [
    (40, 32, 12, False, 1, 1, 1),
    (40, 32, 12, True, 1, 1, 1),
    (40, 32, 12, False, 16, 9, 2),
    (40, 32, 12, True, 16, 9, 2),
    (40, 32, 12, True, 16, 9, 1),
    (600, 128, 20, True, 8, 5, 2),
    (40, 120, 20, False, 8, 5, 2),       # groups that do not end with lanes
    (40, 384, 40, True, 1, 1, 1),
    (40, 1024, 64, True, 32, 9, 2),
]


@pytest.mark.parametrize("shape", SHAPES, ids=[str(i) for i in range(len(SHAPES))])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_far_logits(shape, renorm, dtype):
    torch, moe = _moe()
    T, E, K, with_bias, groups, top_groups, group_top = shape
    log("route far logits %s renorm=%s %s" % (shape, renorm, dtype))
    x = _far_logits(torch, T, E, dtype, E + K)
    bias = torch.randn(E, generator=torch.Generator().manual_seed(3)) * 0.05 if with_bias else None
    kw = dict(groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm)
    want_w, want_ids, s = ref.route(x.double().numpy(), K, "sigmoid", bias=None if bias is None else bias.numpy(), **kw)
    leaf = x.cuda().requires_grad_()
    w, ids = moe.route(leaf, K, scores="sigmoid", bias=None if bias is None else bias.cuda(), **kw)
    assert np.array_equal(to_host(ids).view(np.int32), want_ids)
    chosen = np.take_along_axis(s, want_ids, 1)
    total = chosen.sum(1, keepdims=True) + 1e-20 if renorm else np.ones((T, 1))
    # ten fp32 operations of an ulp or two (2^-23), and every score off by FLUSH
    tol = 16 * 2.0 ** -23 * want_w + FLUSH * (1 + K * want_w) / total + FLUSH
    assert np.all(np.abs(w.detach().cpu().double().numpy() - want_w) <= tol)
    dw = torch.randn((T, K), generator=torch.Generator().manual_seed(4))
    got = torch.autograd.grad(w, leaf, dw.cuda())[0].cpu().double().numpy()
    want = ref.route_backward(x.double().numpy(), want_ids, dw.numpy(), "sigmoid", renorm)
    size = np.abs(want).max(1, keepdims=True) + (np.abs(dw.numpy()) * want_w).max(1, keepdims=True)
    # e / (1 + e)^2 of each expert off by FLUSH, times (dw - <dw, w>) / total
    flush = FLUSH * (2 * np.abs(dw.numpy()).max(1, keepdims=True) / total + 1)
    tol = torch.finfo(x.dtype).eps / 2 * np.abs(want) + 64 * 2.0 ** -23 * size + flush
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("value", [-88.5, -88.75, -89.0, -90.5, -92.5, -95.0, -97.0, -99.0, -100.0, -101.0, -103.9, -104.5])
def test_one_far_logit(value):
    """A group of {5, value} is worth about 1, and a far expert's choice is its bias."""
    torch, moe = _moe()
    x = torch.full((1, 8), value)
    x[0, 2] = 5.0
    x[0, 4:] = torch.tensor([-1.0, -1.25, -2.0, -2.5])
    w, ids = moe.route(x.cuda(), 2, scores="sigmoid", groups=4, top_groups=1, group_top=2)
    # groups {~0, ~0}, {0.993, ~0}, {0.269, 0.223}, {0.119, 0.076}
    assert ids.tolist() == [[2, 3]] and torch.isfinite(w).all()
    assert abs(float(w[0, 0]) - 1.0) <= 2.0 ** -22 and float(w[0, 1]) <= 1e-30
    bias = torch.zeros(8)
    bias[1] = 0.75
    w, ids = moe.route(x.cuda(), 2, scores="sigmoid", bias=bias.cuda(), renormalize=False)
    assert ids.tolist() == [[2, 1]] and 0.0 <= float(w[0, 1]) <= 1e-37
