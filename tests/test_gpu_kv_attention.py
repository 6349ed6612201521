"""Attention over the paged MXFP4 cache against its definition in 64 bits."""

import math

import numpy as np
import pytest

import kv_util as ref
from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def _kv():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    return torch, kvcache


class Case:
    """A filled cache with a shuffled table, and its values in 64 bits."""

    def __init__(self, lengths, queries, heads, kv_heads, d, page, seed=0, spread=1.0, garbage=None):
        torch, kvcache = _kv()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lengths, self.queries, self.page, self.d = lengths, queries, page, d
        need = [ref.pages_of(max(n, 0), page) for n in lengths]
        pages = sum(need) + 2
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        width = max(need + [1]) + 1
        self.table = torch.full((len(lengths), width), -1, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.cache = kvcache.new(pages, page, kv_heads, d, device="cuda")
        k, v = ((torch.randn((pages * page, kv_heads, d), generator=g, device="cuda") * spread).bfloat16() for _ in range(2))
        if spread != 1.0:
            v = (v.float() / spread).bfloat16()
        kvcache.append(self.cache, k, v, torch.arange(pages * page, dtype=torch.int32, device="cuda"))
        self.k, self.v = ref.cache_values(self.cache, page, d)
        t = sum(queries)
        self.q = torch.randn((t, heads, d), generator=g, device="cuda").bfloat16()
        self.offsets = [0]
        for n in queries:
            self.offsets.append(self.offsets[-1] + n)
        if garbage is not None:      # every byte of places behind the sequences
            self._fill(garbage)
        self.torch, self.kvcache = torch, kvcache

    def _fill(self, byte):
        page, d = self.page, self.d
        half, few = page * d // 2, page * d // 32
        used = {}
        for b, n in enumerate(self.lengths):
            for j in range(ref.pages_of(max(n, 0), page)):
                used[int(self.table[b, j])] = min(page, n - j * page)
        for p in range(self.cache.shape[0]):
            n = used.get(p, 0)
            r = self.cache[p]
            r[:, :half].view(-1, page, d // 2)[:, n:] = byte
            v = r[:, half:2 * half].view(-1, page // 4, d // 8, 4, 4)
            for i in range(n, page):
                v[:, i // 4, :, i % 4] = byte
            r[:, 2 * half:2 * half + few].view(-1, page, d // 32)[:, n:] = byte
            r[:, 2 * half + few:].view(-1, d // 32, page)[..., n:] = byte

    def i32(self, values):
        return self.torch.tensor(values, dtype=self.torch.int32, device="cuda")

    def run(self, offsets="own", **kw):
        offsets = self.i32(self.offsets) if isinstance(offsets, str) else offsets
        return self.kvcache.attention(self.q, self.cache, self.table, self.i32(self.lengths), offsets, lse=True, **kw)

    def check(self, got, scale=None, window=0, label=""):
        torch = self.torch
        scale = self.d ** -0.5 if scale is None else scale
        out, lse, bound, lse_bound = ref.attention(self.q, self.k, self.v, self.page, self.table, self.lengths, self.offsets, scale, window)
        o, l = got
        bad = ~((o.double() - out).abs() <= bound)
        assert not bool(bad.any()), "%s: %d of %d outputs off, the worst by %.2f of its bound" % (
            label, int(bad.sum()), bad.numel(), float(((o.double() - out).abs() / bound)[bad].nan_to_num(1e9).max()))
        empty = torch.isinf(lse)
        assert torch.equal(torch.isinf(l) & (l < 0), empty), label
        off = torch.where(empty, 0.0, (l.double() - lse).abs())
        assert bool((off <= lse_bound).all()), "%s: lse off by %.3g (bound %.3g)" % (label, float(off.max()), float(lse_bound.max()))
        assert bool((o[empty] == 0).all()), label


HEADS = [(1, 1), (3, 3), (8, 2), (14, 2), (16, 1)]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", HEADS)
@pytest.mark.parametrize("page", [16, 64])
def test_one_query_each(d, heads, kv_heads, page):
    lengths = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 0, 300, 1025]
    log("one query D=%d heads=%d/%d page=%d" % (d, heads, kv_heads, page))
    c = Case(lengths, [1] * len(lengths), heads, kv_heads, d, page, seed=heads + d)
    c.check(c.run(offsets=None), label="without offsets")
    c.check(c.run(max_queries=1), label="with offsets")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("heads,kv_heads", [(4, 4), (8, 2), (5, 1), (40, 2)])
def test_few_and_many_queries(d, heads, kv_heads):
    """Runs of 0 to 200 queries, at every place of a tile; the kernel for few queries and the one for many."""
    queries = [0, 1, 2, 7, 16, 0, 33, 64, 65, 131, 200, 3]
    lengths = [40, 1, 2, 70, 16, 0, 500, 64, 66, 131, 777, 1000]
    log("queries D=%d heads=%d/%d" % (d, heads, kv_heads))
    c = Case(lengths, queries, heads, kv_heads, d, 32, seed=d + heads)
    for most in (200, 1, 4, None):
        c.check(c.run(max_queries=most), label="max_queries %s" % most)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 1000, 2 ** 40])
def test_window(d, window):
    queries, lengths = [1, 5, 150, 1], [513, 200, 400, 20]
    log("window %d D=%d" % (window, d))
    c = Case(lengths, queries, 4, 2, d, 16, seed=window % 1000)
    for most in (150, 1):
        c.check(c.run(max_queries=most, window=window), window=window, label="max_queries %d" % most)


@pytest.mark.parametrize("most", [1, 300])
def test_more_queries_than_keys(most):
    """Queries in front of the first key see nothing: zeros, and -inf."""
    log("more queries than keys, max_queries %d" % most)
    c = Case([0, 3, 40, 0, 100, -5], [2, 9, 70, 0, 300, 4], 4, 2, 128, 16, seed=3)
    c.check(c.run(max_queries=most))
    c.check(c.run(max_queries=most, window=5), window=5)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("d", [64, 256])
def test_pages(page, d):
    c = Case([1000, 255, 257, 31], [3, 255, 100, 31], 2, 1, d, page, seed=page)
    log("page %d D=%d" % (page, d))
    for most in (255, 1):
        c.check(c.run(max_queries=most))


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("queries", [1, 3, 40])
def test_a_long_sequence_in_parts(d, queries):
    """Long contexts, whose keys are cut into parts that a second launch joins; short ones beside them."""
    torch, kvcache = _kv()
    lengths, runs = [20011, 100, 7000, 0, 513], [queries, 1, queries, 1, queries]
    log("parts D=%d queries=%d" % (d, queries))
    c = Case(lengths, runs, 8, 2, d, 64, seed=queries)
    width, t = c.table.shape[1], sum(runs)
    assert kvcache.kv_attention_workspace_bytes(t, 8, 2, d, 5, width, 64, 1, queries, 0) > 0
    first = c.run(max_queries=queries)
    c.check(first)
    for _ in range(3):        # from run to run the same bits
        again = c.run(max_queries=queries)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    c.check(c.run(max_queries=queries, window=3000), window=3000)


@pytest.mark.parametrize("byte", [0xFF, 0x7F])
@pytest.mark.parametrize("most", [1, 90])
def test_what_stands_behind_a_sequence_does_not_matter(byte, most):
    """Places that no query sees hold codes and scales of NaN, or of huge values: the same bits come out."""
    torch, _ = _kv()
    lengths, queries = [1, 18, 63, 200, 333], [1, 3, 1, 90, 2]
    for d in (64, 128, 256):
        a, b = (Case(lengths, queries, 4, 2, d, 32, seed=1, garbage=x) for x in (None, byte))
        assert not torch.equal(a.cache, b.cache)
        for x, y in zip(a.run(max_queries=most), b.run(max_queries=most)):
            assert torch.equal(x, y)


def test_queries_do_not_see_each_other():
    """A NaN query, and one of infinities, spoil their own rows alone."""
    torch, _ = _kv()
    for most in (1, 200):
        c = Case([300, 250], [200, 4], 4, 2, 128, 32, seed=8)
        want = c.run(max_queries=most)
        c.q[17, 1] = math.nan
        c.q[203, 2, 5] = math.inf
        got = c.run(max_queries=most)
        touched = torch.zeros((204, 4), dtype=torch.bool, device="cuda")
        touched[17, 1] = touched[203, 2] = True
        for x, y in zip(got, want):
            assert torch.equal(x[~touched], y[~touched])
        assert bool(got[0][17, 1].isnan().all())


@pytest.mark.parametrize("most", [1, 100])
def test_numbers_that_are_no_page(most):
    """Keys of such pages are not there."""
    c = Case([200, 90, 500], [1, 40, 100], 4, 2, 128, 16, seed=5)
    c.table[0, 3] = -1
    c.table[0, 12] = 10 ** 6
    c.table[1, :] = -7
    c.table[2, ::2] = 2 ** 31 - 1
    log("no pages, max_queries %d" % most)
    c.check(c.run(max_queries=most))


def test_lengths_past_the_table():
    torch, kvcache = _kv()
    c = Case([64, 64], [1, 2], 2, 2, 64, 16, seed=6)
    c.table = c.table[:, :4]
    want = c.run()
    c.lengths = [2 ** 31 - 1, 70]
    got = c.run()
    for x, y in zip(got, want):
        assert torch.equal(x, y)
    empty = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    o, l = kvcache.attention(c.q, c.cache, empty, c.i32([5, 6]), c.i32([0, 1, 3]), lse=True)
    assert bool((o == 0).all()) and bool((l == -math.inf).all())


@pytest.mark.parametrize("long", [False, True])
@pytest.mark.parametrize("most", [1, 50])
def test_rows_of_no_sequence_are_left(long, most):
    torch, kvcache = _kv()
    queries = [3, 50, 1]
    c = Case([40, 9000 if long else 90, 7], queries, 4, 2, 128, 16, seed=7)
    want = c.run(max_queries=most)[0]
    t = sum(queries)
    q = torch.cat((torch.randn((5, 4, 128), device="cuda").bfloat16(), c.q, torch.randn((9, 4, 128), device="cuda").bfloat16()))
    out = torch.full((t + 14, 4, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    got = kvcache.attention(q, c.cache, c.table, c.i32(c.lengths), c.i32([5 + x for x in c.offsets]), max_queries=most, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(out[5:5 + t], want) and bool((out[:5] == 7).all()) and bool((out[5 + t:] == 7).all())


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-4, 2, 100, 9], [9, 5, 2, 0], [0, 0, 0, 0], [2 ** 31 - 1, 0, 5, 6], [0, 9, 9, 9]])
@pytest.mark.parametrize("most", [1, 60])
def test_odd_offsets(offsets, most):
    """Offsets that do not rise, or leave the rows: clamped, and raised to the running maximum."""
    torch, kvcache = _kv()
    log("offsets %s max_queries %d" % (offsets, most))
    c = Case([50, 60, 70], [3, 3, 3], 2, 1, 64, 16, seed=9)
    out = torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kvcache.attention(c.q, c.cache, c.table, c.i32(c.lengths), c.i32(offsets), max_queries=most, out=out)
    clamped, top = [], 0
    for x in offsets:
        top = max(top, min(max(x, 0), 9))
        clamped.append(top)
    c.offsets = clamped
    want, _, bound, _ = ref.attention(c.q, c.k, c.v, 16, c.table, c.lengths, clamped, 64 ** -0.5, 0)
    rows = ~want.isnan().all(2).all(1)
    assert bool(((out.double() - want).abs() <= bound)[rows].all()) and bool((out[~rows] == 7).all())


def test_no_rows_and_no_sequences():
    torch, kvcache = _kv()
    cache = kvcache.new(2, 16, 2, 64, device="cuda")
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert kvcache.attention(q, cache, torch.zeros((0, 3), dtype=torch.int32, device="cuda"), i).shape == (0, 4, 64)
    lengths = torch.ones(3, dtype=torch.int32, device="cuda")
    o, l = kvcache.attention(q, cache, torch.zeros((3, 3), dtype=torch.int32, device="cuda"), lengths,
                             torch.zeros(4, dtype=torch.int32, device="cuda"), lse=True)
    assert o.shape == (0, 4, 64) and l.shape == (0, 4)


def test_strides_of_queries():
    torch, kvcache = _kv()
    c = Case([100, 300], [1, 60], 4, 2, 128, 16, seed=10)
    want = c.run()
    packed = torch.randn((61, 10, 128), device="cuda").bfloat16()
    packed[:, 3:7] = c.q
    c.q = packed[:, 3:7]
    for x, y in zip(c.run(), want):
        assert torch.equal(x, y)
    c.q = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    for x, y in zip(c.run(), want):
        assert torch.equal(x, y)
    wide = torch.full((2, c.table.shape[1] + 7), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    for x, y in zip(c.run(), want):
        assert torch.equal(x, y)


@pytest.mark.parametrize("scale", [1e-4, 0.5, 3.0])
@pytest.mark.parametrize("most", [1, 70])
def test_scale(scale, most):
    """From an even average to a softmax of one key."""
    c = Case([400, 333], [2, 70], 4, 2, 64, 32, seed=12)
    c.check(c.run(max_queries=most, scale=scale), scale=scale)


@pytest.mark.parametrize("most", [1, 70])
def test_large_and_small_queries(most):
    """Queries of every magnitude, with parts far below their largest value, and zeros."""
    torch, _ = _kv()
    c = Case([400, 333], [8, 70], 4, 2, 128, 32, seed=13)
    g = torch.Generator(device="cuda").manual_seed(1)
    power = torch.randint(-30, 3, c.q.shape, generator=g, device="cuda").float()
    c.q = (c.q.float() * torch.exp2(power)).bfloat16()
    c.q[3] = 0
    c.q[5, 1] = (c.q[5, 1].float() * 2.0 ** -90).bfloat16()
    c.check(c.run(max_queries=most))


def test_growing_scores_rescale():
    """Scores that grow along the keys by far more than any allowance for a late maximum."""
    torch, kvcache = _kv()
    for d in (64, 128, 256):
        c = Case([1500], [1], 2, 1, d, 16, seed=14)
        slots = (c.table[0, :, None] * 16 + torch.arange(16, device="cuda")).reshape(-1)[:1500].to(torch.int32)
        ramp = torch.linspace(-3, 3, 1500, device="cuda")[:, None, None]
        k = (c.q[0, 0] * ramp).expand(1500, 1, d).bfloat16()
        v = torch.randn((1500, 1, d), device="cuda").bfloat16()
        for order in (slots, slots.flip(0)):
            kvcache.append(c.cache, k, v, order)
            c.k, c.v = ref.cache_values(c.cache, 16, d)
            for most in (1, 64):
                c.q = c.q[:1].expand(1, 2, d).contiguous()
                c.check(c.run(max_queries=most), label="D=%d most=%d" % (d, most))


def test_drawn_sizes():
    """Seeded random sizes, heads, pages, windows and runs."""
    rng = np.random.default_rng(20)
    for i in range(40):
        d, page = int(rng.choice([64, 128, 256])), int(rng.choice([16, 32, 64, 128]))
        kv_heads, group = int(rng.integers(1, 4)), int(rng.choice([1, 2, 3, 6, 8, 16, 17]))
        n = int(rng.integers(1, 7))
        lengths = [int(x) for x in rng.integers(0, 900, n)]
        queries = [int(x) for x in (rng.integers(0, 6, n) if rng.random() < 0.5 else rng.integers(0, 90, n))]
        window = int(rng.choice([0, 0, int(rng.integers(1, 500))]))
        log("drawn %d: D=%d page=%d heads=%dx%d lengths=%s queries=%s window=%d" % (i, d, page, kv_heads, group, lengths, queries, window))
        if sum(queries) == 0:
            continue
        c = Case(lengths, queries, kv_heads * group, kv_heads, d, page, seed=i)
        c.check(c.run(window=window, max_queries=max(max(queries), 1)), window=window, label="drawn %d" % i)


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [0, 9, 2, 4], [2, 7, 7, 1], [-4, 2, 100, 9]])
@pytest.mark.parametrize("most", [3, 60])
def test_odd_offsets_in_parts(offsets, most):
    """The same where the keys are cut into parts: the joining launch holds the same rows for a sequence's."""
    torch, kvcache = _kv()
    log("offsets %s max_queries %d" % (offsets, most))
    c = Case([5000, 60, 4000], [3, 3, 3], 2, 1, 64, 16, seed=10)
    assert kvcache.kv_attention_workspace_bytes(9, 2, 1, 64, 3, c.table.shape[1], 16, 1, most, 0) > 0
    out = torch.full((9, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    kvcache.attention(c.q, c.cache, c.table, c.i32(c.lengths), c.i32(offsets), max_queries=most, out=out)
    clamped, top = [], 0
    for x in offsets:
        top = max(top, min(max(x, 0), 9))
        clamped.append(top)
    want, _, bound, _ = ref.attention(c.q, c.k, c.v, 16, c.table, c.lengths, clamped, 64 ** -0.5, 0)
    rows = ~want.isnan().all(2).all(1)
    assert bool(((out.double() - want).abs() <= bound)[rows].all()) and bool((out[~rows] == 7).all())


def test_as_many_sequences_and_heads_as_fit():
    """2^24 rows of single queries: every sequence has the same page and query, and gets the same answer."""
    torch, kvcache = _kv()
    c = Case([13], [1], 128, 8, 64, 16, seed=11)
    n = 1 << 17
    log("%d sequences of %d heads" % (n, 128))
    o, l = kvcache.attention(c.q.expand(n, 128, 64), c.cache, c.table.expand(n, -1).contiguous(), c.i32([13]).expand(n).contiguous(),
                             lse=True)
    want, lse = c.run(offsets=None)
    assert bool((o == want).all()) and bool((l == lse).all())


def test_windows_past_every_length():
    """Windows that no sequence is as long as, up to the largest number: none."""
    torch, kvcache = _kv()
    c = Case([20011, 70], [2, 1], 4, 2, 128, 64, seed=12)
    want = c.run(max_queries=2)
    for window in (1 << 20, 2 ** 31 - 1, 2 ** 31, 2 ** 63 - 1):
        for x, y in zip(c.run(max_queries=2, window=window), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("heads,kv_heads,most", [(8, 2, 9), (8, 2, 16), (3, 3, 33), (3, 3, 64), (7, 1, 9), (60, 1, 1)])
def test_between_few_and_many_rows(d, page, heads, kv_heads, most):
    """33 to 64 rows of a sequence and head; runs longer than announced; windows; a long context in parts."""
    queries = [most, 1, max(most - 3, 1), 2 * most + 1, most]
    lengths = [700, 130, 40, 333, 5000]
    log("D=%d page=%d heads %d/%d queries %s" % (d, page, heads, kv_heads, queries))
    c = Case(lengths, queries, heads, kv_heads, d, page, seed=most + d)
    c.check(c.run(max_queries=most))
    c.check(c.run(max_queries=most, window=77), window=77)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("queries", [1, 5, 40])
@pytest.mark.parametrize("longest", [1100, 2000, 4000])
def test_few_parts(d, queries, longest):
    """Two to eight parts, which one wave of a row joins; rows in front of the sequences and behind them stay."""
    torch, kvcache = _kv()
    runs = [queries, 1, queries, 2, 1]
    log("D=%d queries=%d longest=%d" % (d, queries, longest))
    c = Case([longest, 7, longest - 600, 0, 530], runs, 6, 2, d, 16, seed=longest + queries)
    t, width = sum(runs), c.table.shape[1]
    size = kvcache.kv_attention_workspace_bytes(t + 8, 6, 2, d, 5, width, 16, 1, queries, 0)
    assert 2 <= size // ((t + 8) * 6 * (d + 2) * 4) <= 8
    first = c.run(max_queries=queries)
    c.check(first)
    c.check(c.run(max_queries=queries, window=900), window=900)
    q = torch.cat((c.q[:3], c.q, c.q[:1].expand(5, -1, -1)))
    out = torch.full((t + 8, 6, d), 7.0, dtype=torch.bfloat16, device="cuda")
    kvcache.attention(q, c.cache, c.table, c.i32(c.lengths), c.i32([3 + x for x in c.offsets]), max_queries=queries, out=out)
    assert torch.equal(out[3:3 + t], first[0]) and bool((out[:3] == 7).all()) and bool((out[3 + t:] == 7).all())
