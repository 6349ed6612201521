"""Sequences longer than their block table: the queries stay at their places at the
end of the sequence, and the keys that the table does not hold are not there."""

import math

import pytest

import kv_util as ref
from gpu_util import log, need_gpu
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


def _widened(torch, table, lengths, page):
    """The same table with an entry for every key, -1 where there was none."""
    width = max(table.shape[1], max(ref.pages_of(max(n, 0), page) for n in lengths))
    wide = torch.full((table.shape[0], width), -1, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = table
    return wide


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("most", [1, 90])
@pytest.mark.parametrize("window", [0, 1, 10, 40, 300])
def test_queries_stay_where_they_are(d, most, window):
    """From one query just behind the table's last key to runs that lie behind it as a whole, or begin inside it."""
    torch = need_gpu()
    queries, lengths = [2, 1, 70, 3, 90, 5, 33], [100, 65, 100, 64, 130, 1000, 66]
    log("D=%d most=%d window=%d" % (d, most, window))
    c = Case(lengths, queries, 4, 2, d, 16, seed=window + d)
    c.table = c.table[:, :4]                       # 64 keys
    got = c.run(max_queries=most, window=window)
    c.table = _widened(torch, c.table, lengths, 16)
    c.check(got, window=window, label="against the definition")
    c.check(c.run(max_queries=most, window=window), window=window, label="with the wider table")


@pytest.mark.parametrize("queries,most", [(1, 1), (6, 6), (200, 200)])
def test_in_parts(queries, most):
    """The same where the keys are cut into parts: the table ends inside the last query's window, or before it."""
    torch = need_gpu()
    lengths = [9000, 9000 + queries // 2, 20000, 8000]
    for window in (0, 1500, 900, 5):
        log("queries=%d window=%d" % (queries, window))
        c = Case(lengths, [queries] * 4, 4, 2, 128, 64, seed=window)
        c.table = c.table[:, :128 + 13]            # 9024 keys
        got = c.run(max_queries=most, window=window)
        c.table = _widened(torch, c.table, lengths, 64)
        c.check(got, window=window)


def test_the_largest_length():
    """2^31 - 1 keys, of which the table holds 64: a query at the end sees them all, with a window none."""
    torch = need_gpu()
    c = Case([64, 64], [3, 70], 4, 2, 64, 16, seed=2)
    narrow, behind = c.table[:, :4], [64 + 3, 64 + 70]
    for most in (1, 70):
        c.table, c.lengths = narrow, [2 ** 31 - 1] * 2
        got = c.run(max_queries=most)
        o, l = c.run(max_queries=most, window=2 ** 31 - 1000)
        assert bool((o == 0).all()) and bool((l == -math.inf).all())
        c.table, c.lengths = _widened(torch, narrow, behind, 16), behind
        c.check(got)
