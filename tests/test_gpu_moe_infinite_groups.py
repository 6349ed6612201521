"""Groups whose two best choices are +inf and -inf (experts forced and barred by
the bias): their value counts as -inf, and never more than top_groups are open."""

import numpy as np
import pytest
import torch

import mx4_util as ref
from gpu_util import log, need_gpu, to_host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("groups,per,T", [(4, 3, 2), (8, 4, 3), (64, 2, 5), (16, 8, 600), (8, 32, 600)])
@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
def test_forced_and_barred(groups, per, T, scores):
    need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    log("infinite groups %d x %d T=%d %s" % (groups, per, T, scores))
    E, inf = groups * per, float("inf")
    g = torch.Generator().manual_seed(groups)
    x = torch.randn((T, E), generator=g)
    bias = torch.zeros((groups, per))
    bias[0::2] = -inf
    bias[0::2, 0] = inf                    # one forced, the others barred
    bias[groups - 1, 1] = inf              # forced and open
    bias = bias.flatten()
    for top_groups in (1, groups // 2, groups - 1):
        kw = dict(groups=groups, top_groups=top_groups, group_top=2)
        K = min(2, top_groups * per)
        with np.errstate(invalid="ignore"):
            _, want, _ = ref.route(x.double().numpy(), K, scores, bias=bias.numpy(), **kw)
        _, ids = moe.route(x.cuda(), K, scores=scores, bias=bias.cuda(), **kw)
        got = to_host(ids).view(np.int32)
        assert np.array_equal(got, want), top_groups
        K = min(64, top_groups * per)
        _, ids = moe.route(x.cuda(), K, scores=scores, bias=bias.cuda(), **kw)
        opened = [len(set(row // per)) for row in to_host(ids).view(np.int32)]
        assert max(opened) <= top_groups
