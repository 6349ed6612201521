"""Tables far wider than the sequences in them, as a program has that admits long requests:
the same answers, from run to run the same bits, and no call refused for a split of the keys
that it could do without."""

import math

import pytest

from gpu_util import log, need_gpu
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


def _widen(torch, c, capacity):
    wide = torch.full((c.table.shape[0], capacity // c.page), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("queries,most", [([1, 1, 1, 1, 1, 1, 1], 1), ([1, 5, 0, 5, 2, 5, 5], 5), ([40, 1, 33, 0, 40, 2, 40], 40),
                                          ([300, 1, 77, 128, 0, 300, 129], 300)])
def test_short_sequences_beside_long_ones(d, queries, most):
    """Sequences of one part, whose outputs are written at once, of two, and of many, in one call."""
    torch = need_gpu()
    lengths = [513, 5, 0, 1025, 17000, 600, 40000]
    log("D=%d queries=%s" % (d, queries))
    c = Case(lengths, queries, 8, 2, d, 64, seed=most + d)
    tight = c.run(max_queries=most)
    c.check(tight, label="table of 40064 keys")
    _widen(torch, c, 1 << 20)
    for window in (0, 900):
        got = c.run(max_queries=most, window=window)
        table, c.table = c.table, c.table[:, :626]     # for the definition the entries behind them say nothing
        c.check(got, window=window, label="table of 2^20 keys, window %d" % window)
        c.table = table
        for _ in range(2):
            for x, y in zip(got, c.run(max_queries=most, window=window)):
                assert torch.equal(x, y)


@pytest.mark.parametrize("most", [1, 60])
def test_what_the_workspace_held_does_not_matter(most):
    """A workspace full of NaN, or of large whole numbers, and rows of no sequence between those of some."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    queries, t = [3, 60, 1, 2], 66
    c = Case([700, 9000, 5, 30000], queries, 4, 2, 128, 64, seed=7)
    _widen(torch, c, 1 << 17)
    want, want_lse = c.run(max_queries=most)
    need = kvcache.kv_attention_workspace_bytes(t + 9, 4, 2, 128, 4, 2048, 64, 1, most, 0)
    assert need > 0
    log("most=%d workspace of %d bytes" % (most, need))
    q = torch.cat((c.q[:4], c.q, c.q[:5]))
    offsets, lengths = c.i32([4 + x for x in c.offsets]), c.i32(c.lengths)
    for word in (0x7FC00000, 0x7FFFFFFF, -1, 0, 3):
        work = torch.full((need // 4,), word, dtype=torch.int32, device="cuda")
        out = torch.full((t + 9, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((t + 9, 4), 7.0, device="cuda")
        kvcache.kv_attention(q, 512, 128, t + 9, 4, c.cache, c.cache.shape[0], 64, 2, 128, c.table, 2048, 2048, lengths, offsets, 4, most,
                             128 ** -0.5, 0, out, lse, work, need)
        for got, x in ((out, want), (lse, want_lse)):
            # (nine more rows may be cut otherwise: the sum's order, of 32 bits)
            assert torch.allclose(got[4:4 + t].float(), x.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
            assert bool((got[:4] == 7).all()) and bool((got[4 + t:] == 7).all())


def test_more_rows_than_a_joining_launch_holds():
    """2^24 queries behind a table of 2^20 keys: one part, no launch that could not be made."""
    torch = need_gpu()
    c = Case([13], [20], 1, 1, 64, 16, seed=11)
    want, lse = c.run(max_queries=20)
    _widen(torch, c, 1 << 20)
    n = 1 << 24
    log("%d queries" % n)
    q = torch.zeros((1, 1, 64), dtype=torch.bfloat16, device="cuda").expand(n, 1, 64).contiguous()
    q[-20:] = c.q
    o, l = c.kvcache.attention(q, c.cache, c.table, c.i32([13]), c.i32([0, n]), lse=True)
    assert torch.allclose(o[-20:].float(), want.float(), rtol=2.0 ** -7, atol=2.0 ** -10)
    assert torch.allclose(l[-13:], lse[-13:], rtol=0, atol=2.0 ** -12)
    assert bool((o[:-13] == 0).all()) and bool((l[:-13] == -math.inf).all())
