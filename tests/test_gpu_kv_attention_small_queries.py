"""Queries near the smallest BF16 numbers against keys near the largest: a query keeps
its bits down to 2^-21 of its row's largest value there too."""

import pytest

from gpu_util import log, need_gpu
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 70])
def test_tiny_queries_and_huge_keys(d, most):
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    import kv_util as ref
    for power in (-100, -107, -112, -116, -120, -124, -128):
        log("D=%d most=%d queries times 2^%d" % (d, most, power))
        c = Case([300, 133], [4, 70], 4, 2, d, 32, seed=3)
        slots = torch.arange(c.cache.shape[0] * 32, dtype=torch.int32, device="cuda")
        g = torch.Generator(device="cuda").manual_seed(5)
        k, v = (torch.randn((slots.numel(), 2, d), generator=g, device="cuda") for _ in range(2))
        # scores of a few units: the query times 2^power, the keys times 2^-power
        up = min(-power, 122)
        kvcache.append(c.cache, torch.ldexp(k, torch.tensor(up, device="cuda")).bfloat16(), v.bfloat16(), slots)
        c.k, c.v = ref.cache_values(c.cache, 32, d)
        c.q = torch.ldexp(c.q.double(), torch.tensor(power, device="cuda")).bfloat16()
        c.check(c.run(max_queries=most, scale=0.5), scale=0.5, label="2^%d" % power)
