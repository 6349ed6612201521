"""The attention layer's steps with heads of 128 and 256 values, and its refusal of gradients."""

import pytest

import test_gpu_attention_layer as base
from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("page", [16, 32])
@pytest.mark.parametrize("window", [0, 24])
def test_steps(monkeypatch, d, page, window):
    log("D=%d page=%d window=%d" % (d, page, window))
    monkeypatch.setattr(base, "D", d)
    monkeypatch.setattr(base, "PAGE", page)
    base.test_steps(window)


def test_a_gradient_is_refused():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    layer, normal = base._layer(torch, 1)
    cache = kvcache.new(4, base.PAGE, base.KV, base.D, device="cuda")
    free, left = kvcache.pool(4, device="cuda")
    table = torch.full((1, 4), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(1, dtype=torch.int32, device="cuda")
    plan = kvcache.extend(table, lengths, lengths + 5, free, left, 5, base.PAGE)
    x = normal(5, base.HIDDEN).bfloat16().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        layer(x, cache, table, plan)
    assert not bool(cache.any())
    with torch.no_grad():
        a = layer(x, cache, table, plan)
    assert not a.requires_grad and torch.equal(a, layer(x.detach(), cache, table, plan))
