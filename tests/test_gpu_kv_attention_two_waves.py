"""The kernel for many queries in workgroups of two waves: 33 to 64 rows of a run and
key-value head, where the heads' tiles times parts of 512 keys are 1024 or more (of
256 values always)."""

import pytest

from gpu_util import log, need_gpu
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu

KV = 8


def _two_waves(kvcache, d, page, width, sequences, tokens, heads, queries, window=0):
    """Whether a call of these sizes is one: with 512 tiles and 1024 to 1535 keys the kernel of 64 rows wants two parts of
    them (1024 workgroups), that of 128 rows one."""
    keys = min(width * page, window + queries) if window else width * page
    assert 33 <= queries * heads // KV <= 64 and sequences * KV * (keys // 512) >= 1024
    return kvcache.kv_attention_workspace_bytes(tokens, heads, KV, d, sequences, width, page, 1, queries, window) > 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads,queries", [(8, 33), (16, 32), (40, 7), (56, 9)])
def test_against_the_definition(d, page, heads, queries):
    """64 sequences of every length to 1400, runs that fill their tile, single queries, and runs longer than announced."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    lengths = [1 + (i * 397) % 1400 for i in range(63)] + [1400]
    runs = [(queries, 1, queries, max(queries - 5, 1), 0)[i % 5] for i in range(64)]
    runs[11] = 2 * queries + 3
    log("D=%d page=%d heads=%d queries=%d" % (d, page, heads, queries))
    c = Case(lengths, runs, heads, KV, d, page, seed=d + queries)
    width = c.table.shape[1]
    for window in (0, 1100):
        assert _two_waves(kvcache, d, page, width, 64, sum(runs), heads, queries, window)
        got = c.run(max_queries=queries, window=window)
        c.check(got, window=window, label="window %d" % window)
        for x, y in zip(got, c.run(max_queries=queries, window=window)):
            assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128])
def test_one_part(d):
    """1024 heads' tiles of a thousand keys: enough workgroups without parts, written as they are."""
    need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    n = 128
    lengths = [(i * 389) % 980 + 1 for i in range(n)]
    c = Case(lengths, [40 - i % 3 for i in range(n)], KV, KV, d, 16, seed=d)
    t, width = sum(c.queries), c.table.shape[1]
    assert width * 16 // 512 == 1 and n * KV >= 1024
    assert kvcache.kv_attention_workspace_bytes(t, KV, KV, d, n, width, 16, 1, 40, 0) == 0
    log("D=%d, %d rows" % (d, t))
    c.check(c.run(max_queries=40))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_four_parts(d, page):
    """Few sequences of 20000 keys: as many parts as give 1024 workgroups; keys that are not there and bytes of NaN behind."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    c = Case([20000, 17, 9001, 4000], [48, 48, 33, 1], KV, KV, d, page, seed=page, garbage=0xFF)
    width = c.table.shape[1]
    assert 4 * KV * min(width * page // 512, 64) >= 1024
    rows = 130 * KV
    assert kvcache.kv_attention_workspace_bytes(130, KV, KV, d, 4, width, page, 1, 48, 0) // (rows * (d + 2) * 4) == 32
    c.table[0, 5] = -1
    c.table[2, 7] = 10 ** 7
    log("D=%d page=%d" % (d, page))
    got = c.run(max_queries=48)
    c.check(got)
    for x, y in zip(got, c.run(max_queries=48)):
        assert torch.equal(x, y)
