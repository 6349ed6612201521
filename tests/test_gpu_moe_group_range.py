"""Groups of experts whose two best choices add up to more than fp32 holds, as
biases of the type's lowest value give them: ordered as in 64 bits."""

import numpy as np
import pytest

import mx4_util as ref
from gpu_util import log, need_gpu, to_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,per,T", [(16, 4, 3), (12, 3, 3), (128, 32, 3), (256, 32, 3), (256, 64, 600), (384, 96, 600)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_sums_past_the_range(E, per, T, scores):
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    log("group sums E=%d per=%d T=%d %s" % (E, per, T, scores))
    low, inf = torch.finfo(torch.float32).min, float("inf")
    groups = E // per
    x = torch.randn((T, E), generator=torch.Generator().manual_seed(E))
    # group 0 open to all, 1 shut by -inf, 2 by the lowest value, the last by a little less
    bias = torch.full((groups, per), -inf)
    bias[0] = 0.0
    bias[2] = low
    bias[groups - 1] = low * 0.75
    bias = bias.flatten()
    for top_groups in (2, 3):
        kw = dict(groups=groups, top_groups=top_groups, group_top=2)
        K = min(top_groups * per, 64)
        _, want, _ = ref.route(x.double().numpy(), K, scores, bias=bias.numpy(), **kw)
        _, ids = moe.route(x.cuda(), K, scores=scores, bias=bias.cuda(), **kw)
        assert np.array_equal(to_host(ids).view(np.int32), want), top_groups
    # the same upwards: both sums past the range, the later group's the larger,
    # every expert's choice far from the next one's
    up = torch.zeros((groups, per))
    spread = 1 - 0.2 * torch.arange(per) / per
    up[1] = -low * 0.75 * spread
    up[groups - 1] = -low * spread
    kw = dict(groups=groups, top_groups=1, group_top=2)
    K = min(per, 64)
    _, want, _ = ref.route(x.double().numpy(), K, scores, bias=up.flatten().numpy(), **kw)
    _, ids = moe.route(x.cuda(), K, scores=scores, bias=up.flatten().cuda(), **kw)
    assert want.min() >= E - per and np.array_equal(to_host(ids).view(np.int32), want)
