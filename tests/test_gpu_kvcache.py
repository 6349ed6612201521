"""Block tables, slots, and the paged MXFP4 cache against plain implementations."""

import numpy as np
import pytest

import kv_util as ref
import mx4_util
from gpu_util import log, need_gpu, to_dev, to_dev_bf16, to_host

pytestmark = pytest.mark.gpu


def _kv():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    return torch, kvcache


def _i32(a):
    return to_dev(np.asarray(a, np.int32))


def _requests(rng, n, page, past, new, width=None, spare=3, short=0):
    """A table in which every request has the pages of its past, and a shuffled stack of the others."""
    lengths, counts = rng.integers(0, past + 1, n), rng.integers(0, new + 1, n)
    held = -(-lengths // page)
    need = -(-(lengths + counts) // page) - held
    width = int(max(1, (held + need).max(initial=1))) if width is None else width
    pages = int(held.sum() + need.sum()) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((n, width), -1, np.int32)
    at = 0
    for b in range(n):
        h = min(int(held[b]), width)
        table[b, :h] = order[at:at + h]
        at += h
    free = np.full(pages, -1, np.int32)
    free[:pages - at] = order[at:]
    return table, lengths.astype(np.int32), counts.astype(np.int32), free, max(0, pages - at - short)


def _check_extend(table, lengths, counts, free, left, tokens, page):
    torch, kvcache = _kv()
    want = ref.extend(table, lengths, counts, free, left, tokens, page)
    t, f = _i32(table), _i32(free)
    got = kvcache.extend(t, _i32(lengths), _i32(counts), f, _i32([left]), tokens, page)
    for name, a, b in zip(got._fields, got, want):
        assert np.array_equal(a.cpu().numpy(), b), name
    assert np.array_equal(t.cpu().numpy(), want[5]) and np.array_equal(f.cpu().numpy(), free)
    return got


@pytest.mark.parametrize("n,page,past,new", [(1, 16, 0, 1), (1, 16, 100, 1), (7, 16, 40, 5), (64, 32, 500, 1), (65, 256, 3000, 700),
                                             (1023, 16, 100, 3), (1024, 64, 10, 80), (1025, 128, 300, 2), (4100, 16, 33, 17),
                                             (3, 16, 50, 30000)])
def test_extend(n, page, past, new):
    rng = np.random.default_rng(n + page)
    table, lengths, counts, free, left = _requests(rng, n, page, past, new)
    total = int(counts.sum())
    log("extend n=%d page=%d past=%d new=%d rows=%d" % (n, page, past, new, total))
    _check_extend(table, lengths, counts, free, left, total, page)
    _check_extend(table, lengths, counts, free, left, total + 1111, page)      # rows of nobody


@pytest.mark.parametrize("short", [1, 5, 60, 10 ** 9])
def test_extend_without_enough_pages(short):
    rng = np.random.default_rng(short % 97)
    table, lengths, counts, free, left = _requests(rng, 300, 16, 60, 40, short=short)
    log("extend with %d pages less" % short)
    got = _check_extend(table, lengths, counts, free, left, int(counts.sum()), 16)
    # three pages were to spare
    assert (got.slots.cpu().numpy() == -1).any() == (short > 3)


def test_extend_refuses_requests_that_do_not_fit():
    rng = np.random.default_rng(5)
    table, lengths, counts, free, left = _requests(rng, 200, 16, 100, 90, spare=400)
    total = int(counts.sum())
    log("extend with a narrow table, with too few rows")
    _check_extend(table[:, :7], lengths, counts, free, left, total, 16)
    _check_extend(table, lengths, counts, free, left, total // 2, 16)
    _check_extend(table, lengths, counts, free, left, 0, 16)


def test_extend_odd_numbers():
    """Negative and huge lengths and counts, numbers that are no page, a wrong count, no requests."""
    log("extend with odd numbers")
    table = np.full((8, 6), -1, np.int32)
    table[:, 0] = [0, 1, -5, 99, 2, 3, 4, 5]
    lengths = np.array([-3, 5, 16, 10, 2 ** 31 - 1, 7, 2 ** 31 - 20, 16], np.int32)
    counts = np.array([4, -7, 2, 3, 5, 0, 19, 40], np.int32)
    free = np.array([7, 8, -2, 60, 9, 10, 11, 12, 13, 14], np.int32)
    for left in (10, 3, -4, 1000):
        for tokens in (0, 9, 73, 100):
            _check_extend(table, lengths, counts, free, left, tokens, 16)
    none = np.zeros(0, np.int32)
    _check_extend(np.zeros((0, 4), np.int32), none, none, free, 5, 6, 16)
    _check_extend(np.zeros((3, 0), np.int32), np.zeros(3, np.int32), np.array([0, 2, 0], np.int32), free, 5, 6, 16)


def test_extend_of_a_table_with_wide_rows():
    torch, kvcache = _kv()
    rng = np.random.default_rng(9)
    table, lengths, counts, free, left = _requests(rng, 40, 16, 90, 30)
    want = ref.extend(table, lengths, counts, free, left, int(counts.sum()), 16)
    wide = torch.full((40, table.shape[1] + 5), 123, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = _i32(table)
    view = wide[:, :table.shape[1]]
    version = wide._version
    got = kvcache.extend(view, _i32(lengths), _i32(counts), _i32(free), _i32([left]), int(counts.sum()), 16)
    assert np.array_equal(view.cpu().numpy(), want[5]) and bool((wide[:, table.shape[1]:] == 123).all())
    assert np.array_equal(got.slots.cpu().numpy(), want[2]) and wide._version > version


@pytest.mark.parametrize("n", [0, 1, 63, 1000, 1025])
@pytest.mark.parametrize("share", [0.0, 0.4, 1.0])
def test_release(n, share):
    torch, kvcache = _kv()
    rng = np.random.default_rng(n)
    table, lengths, _, free, left = _requests(rng, n, 16, 200, 0)
    if n > 10:
        table[3, :2] = [-1, 10 ** 6]      # no pages
        lengths[5] = -4
        lengths[6] = 10 ** 9              # longer than the table
    finished = rng.random(n) < share
    log("release n=%d share=%s" % (n, share))
    want = ref.release(table, lengths, finished, free, left, 16)
    t, f = _i32(table), _i32(free)
    got = kvcache.release(t, _i32(lengths), to_dev(finished), f, _i32([left]), 16)
    for a, b in zip((*got, t, f), want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_pages_come_back():
    """Steps of growing and leaving requests: no page belongs to two, none is lost."""
    torch, kvcache = _kv()
    rng = np.random.default_rng(11)
    n, page, pages = 37, 16, 300
    table = torch.full((n, 12), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
    free, left = kvcache.pool(pages, device="cuda")
    for step in range(12):
        counts = _i32(rng.integers(0, 30, n))
        plan = kvcache.extend(table, lengths, counts, free, left, 1200, page)
        lengths, left = plan.lengths, plan.free_count
        used = table[table >= 0].cpu().numpy()
        stack = free[:int(left)].cpu().numpy()
        assert sorted(np.concatenate((used, stack)).tolist()) == list(range(pages)), step
        slots = plan.slots[plan.slots >= 0]
        assert slots.unique().numel() == slots.numel()
        lengths, left = kvcache.release(table, lengths, to_dev(rng.random(n) < 0.3), free, left, page)
    lengths, left = kvcache.release(table, lengths, torch.ones(n, dtype=torch.bool, device="cuda"), free, left, page)
    assert int(left) == pages and sorted(free.tolist()) == list(range(pages)) and bool((table == -1).all())


# ------------------------------------------------------------- append and read

def _slots(rng, tokens, pages, page):
    return rng.permutation(pages * page)[:tokens].astype(np.int32)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,heads,page,in_order", [(1, 1, 16, True), (3, 5, 16, False), (64, 8, 32, False), (65, 3, 64, True),
                                                        (257, 2, 256, False), (1000, 1, 128, True)])
def test_append_and_read(d, tokens, heads, page, in_order):
    torch, kvcache = _kv()
    rng = np.random.default_rng(tokens + d)
    pages = -(-tokens // page) + 2
    bits = [mx4_util.heavy_bits((tokens, heads * d), tokens + i).reshape(tokens, heads, d) for i in range(2)]
    slots = np.arange(7, 7 + tokens, dtype=np.int32) if in_order else _slots(rng, tokens, pages, page)
    slots[tokens // 2::9] = np.resize([-1, pages * page, -2 ** 31, 2 ** 31 - 1], slots[tokens // 2::9].size)
    log("append D=%d tokens=%d heads=%d page=%d" % (d, tokens, heads, page))
    before = rng.integers(0, 256, (pages, heads, page * (d + d // 16)), dtype=np.uint8)
    cache = to_dev(before.copy())
    assert kvcache.append(cache, to_dev_bf16(bits[0]), to_dev_bf16(bits[1]), _i32(slots)) is None
    # the expected bytes: the tokens' records put where their slots say
    full = [np.zeros((pages * page, heads, d), np.uint16) for _ in range(2)]
    kept = (slots >= 0) & (slots < pages * page)
    for f, b in zip(full, bits):
        f[slots[kept]] = b[kept]
    want = ref.cache_bytes(*(f.reshape(pages, page, heads, d).transpose(0, 2, 1, 3) for f in full))
    hit = np.zeros((pages * page, heads, d), np.uint16)
    hit[slots[kept]] = 0x3F80     # codes and scales of ones: which bytes a written token has
    mark = [ref.cache_bytes(x, x) for x in (np.broadcast_to(hit.reshape(pages, page, heads, d).transpose(0, 2, 1, 3), (pages, heads, page, d)),)][0]
    expected = np.where(mark != 0, want, before)
    assert np.array_equal(cache.cpu().numpy(), expected)
    k, v = kvcache.read(cache, _i32(slots), d)
    values = [mx4_util.dequantize(*mx4_util.quantize(b.reshape(-1, d))).reshape(tokens, heads, d) for b in bits]
    for got, x in zip((k, v), values):
        assert np.array_equal(mx4_util.bf16_values(to_host(got)), np.where(kept[:, None, None], x, 0.0))


def test_append_of_a_packed_projection():
    """Keys and values as views of one tensor, with strides of their own; head-major ones too."""
    torch, kvcache = _kv()
    t, h, d = 21, 4, 128
    x = torch.randn((t, 3 * h, d), device="cuda").bfloat16()
    k, v = x[:, h:2 * h], x[:, 2 * h:]
    slots = torch.randperm(64, device="cuda")[:t].to(torch.int32)
    a, b, c = (kvcache.new(4, 16, h, d, device="cuda") for _ in range(3))
    kvcache.append(a, k, v, slots)
    kvcache.append(b, k.contiguous(), v.contiguous(), slots)
    kvcache.append(c, k.transpose(0, 1).contiguous().transpose(0, 1), v, slots)
    assert torch.equal(a, b) and torch.equal(a, c) and bool(a.any())
    one = kvcache.new(4, 16, 1, d, device="cuda")
    kvcache.append(one, x[:1, :1].expand(1, 1, d), x[:1, 1:2], slots[:1])
    assert torch.equal(kvcache.read(one, slots[:1], d)[0], kvcache.read(a, slots[:1], d)[0][:, :1]) is False


def test_append_of_values_that_are_not_finite():
    """Infinities and NaN leave finite values in their blocks, and other blocks alone."""
    torch, kvcache = _kv()
    x = torch.randn((4, 2, 64), device="cuda").bfloat16()
    bad = x.clone()
    for i, value in enumerate((float("inf"), float("-inf"), float("nan"), 3.3e38)):
        bad[i, 0, 5] = value
    slots = torch.arange(4, device="cuda", dtype=torch.int32)
    clean, cache = (kvcache.new(1, 16, 2, 64, device="cuda") for _ in range(2))
    kvcache.append(clean, x, x, slots)
    kvcache.append(cache, bad, bad, slots)
    for got, want in zip(kvcache.read(cache, slots, 64), kvcache.read(clean, slots, 64)):
        assert bool(torch.isfinite(got).all())
        assert torch.equal(got[:, 0, 32:], want[:, 0, 32:]) and torch.equal(got[:, 1], want[:, 1])


def test_cache_past_four_gigabytes():
    """Pages on both sides of byte 2^32 of a cache, tables and attention among them."""
    torch, kvcache = _kv()
    h, d, page = 8, 128, 128
    record = h * page * (d + d // 16)
    pages = 2 ** 32 // record + 40
    log("cache of %.2f GB" % (pages * record / 1e9))
    cache = torch.empty((pages, h, page * (d + d // 16)), dtype=torch.uint8, device="cuda")
    chosen = torch.tensor([0, pages - 1, 2 ** 32 // record, 2 ** 32 // record + 1, 3], device="cuda")
    t = chosen.numel() * page
    slots = (chosen[:, None] * page + torch.arange(page, device="cuda")).reshape(-1).to(torch.int32)
    k, v = (torch.randn((t, h, d), device="cuda").bfloat16() for _ in range(2))
    kvcache.append(cache, k, v, slots)
    small = kvcache.new(chosen.numel(), page, h, d, device="cuda")
    kvcache.append(small, k, v, torch.arange(t, device="cuda", dtype=torch.int32))
    assert torch.equal(cache[chosen], small)
    for a, b in zip(kvcache.read(cache, slots, d), kvcache.read(small, torch.arange(t, device="cuda", dtype=torch.int32), d)):
        assert torch.equal(a, b)
    lengths = torch.tensor([t - 3], dtype=torch.int32, device="cuda")
    few = torch.arange(chosen.numel(), device="cuda", dtype=torch.int32)[None]
    for queries in (1, 150):
        q = torch.randn((queries, 2 * h, d), device="cuda").bfloat16()
        offsets = torch.tensor([0, queries], dtype=torch.int32, device="cuda")
        assert torch.equal(kvcache.attention(q, cache, chosen[None].to(torch.int32), lengths, offsets),
                           kvcache.attention(q, small, few, lengths, offsets))


# -------------------------------------------------------------------- refusals

def test_refusals():
    torch, kvcache = _kv()
    log("refusals of the key-value cache")
    cache = kvcache.new(4, 16, 2, 64, device="cuda")
    x = torch.zeros((3, 2, 64), device="cuda", dtype=torch.bfloat16)
    slots = torch.zeros(3, device="cuda", dtype=torch.int32)
    bad_append = [(cache.float(), x, x, slots), (cache[0], x, x, slots), (cache[:, :, :-1], x, x, slots), (cache, x.float(), x, slots),
                  (cache, x[0], x, slots), (cache, x, x[:2], slots), (cache, x[:, :1], x[:, :1], slots), (cache, x, x, slots.long()),
                  (cache, x, x, slots[:2]), (cache, x.transpose(1, 2), x, slots), (cache, x.cpu(), x, slots), (cache, x, x, slots.cpu()),
                  (cache, torch.zeros((3, 2, 96), device="cuda", dtype=torch.bfloat16), x, slots),
                  (cache.transpose(0, 1), x, x, slots), (cache[:, :, ::2], x, x, slots),
                  (torch.zeros((4, 2, 8 * 68), dtype=torch.uint8, device="cuda"), x, x, slots)]
    for args in bad_append:
        with pytest.raises(ValueError):
            kvcache.append(*args)
    with pytest.raises(ValueError, match="gradient"):
        kvcache.append(cache, x.clone().requires_grad_(), x, slots)
    with torch.no_grad():
        kvcache.append(cache, x.clone().requires_grad_(), x, slots[:3] - 1)
    odd = torch.zeros((3, 2, 65), device="cuda", dtype=torch.bfloat16)
    import mxfp8_block_scaled_quantize_amd as mx
    with pytest.raises(mx.MXFP8Error, match="MISALIGNED"):
        kvcache.append(cache, odd[:, :, 1:], odd[:, :, :64], slots)
    for args in ((cache, slots, 96), (cache, slots[None], 64), (cache, slots.float(), 64), (cache, slots, 128)):
        with pytest.raises(ValueError):
            kvcache.read(*args)
    table = torch.zeros((3, 4), device="cuda", dtype=torch.int32)
    q = torch.zeros((3, 4, 64), device="cuda", dtype=torch.bfloat16)
    offsets = torch.arange(4, device="cuda", dtype=torch.int32)

    def attention(q=q, cache=cache, table=table, lengths=slots, offsets=None, **kw):
        return kvcache.attention(q, cache, table, lengths, offsets, **kw)
    attention()
    for bad in (dict(q=q[:2]), dict(q=q[:, :3]), dict(q=q.float()), dict(q=q[0]), dict(q=q.cpu()), dict(q=q[..., ::2]), dict(table=table[:2]),
                dict(table=table.long()), dict(table=table.t()), dict(table=table[0]), dict(table=table.cpu()), dict(lengths=slots.long()),
                dict(lengths=slots[None]), dict(offsets=offsets[:3]), dict(offsets=offsets.long()), dict(scale=0.0), dict(scale=-1.0),
                dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-60), dict(window=-1), dict(max_queries=0),
                dict(out=q.float()), dict(out=q[:2]), dict(out=q.transpose(0, 1)), dict(cache=cache[..., :-4])):
        with pytest.raises(ValueError):
            attention(**bad)
    for bad in (dict(window=1.5), dict(scale="x"), dict(max_queries=2.0), dict(out=3)):
        with pytest.raises(TypeError):
            attention(**bad)
    with pytest.raises(ValueError, match="gradient"):
        attention(q=q.clone().requires_grad_())
    with pytest.raises(ValueError, match="gradient"):
        attention(out=torch.zeros_like(q).requires_grad_())
    out = torch.zeros_like(q)
    version = out._version
    assert attention(out=out) is not None and out._version > version
    free, count = kvcache.pool(8, device="cuda")
    for args in ((table, slots.long(), slots, free, count, 4, 16), (table[:2], slots, slots, free, count, 4, 16),
                 (table, slots, slots[:2], free, count, 4, 16), (table, slots, slots, free.long(), count, 4, 16),
                 (table, slots, slots, free, free, 4, 16), (table, slots, slots, free, count, -1, 16),
                 (table.t(), slots, slots, free, count, 4, 16), (table, slots, slots, free, count, 2 ** 31 - 1, 16)):
        with pytest.raises(ValueError):
            kvcache.extend(*args)
    with pytest.raises(mx.MXFP8Error, match="SHAPE"):
        kvcache.extend(table, slots, slots, free, count, 4, 24)
    for args in ((table, slots, slots, free, count, 16), (table, slots, slots.bool()[:2], free, count, 16)):
        with pytest.raises(ValueError):
            kvcache.release(*args)


def test_forward_mode():
    torch, kvcache = _kv()
    import torch.autograd.forward_ad as fwad
    cache = kvcache.new(2, 16, 1, 64, device="cuda")
    x = torch.zeros((2, 1, 64), device="cuda", dtype=torch.bfloat16)
    slots = torch.zeros(2, device="cuda", dtype=torch.int32)
    table = torch.zeros((2, 2), device="cuda", dtype=torch.int32)
    with fwad.dual_level():
        dual = fwad.make_dual(x, torch.ones_like(x))
        for call in (lambda: kvcache.append(cache, dual, x, slots), lambda: kvcache.append(cache, x, dual, slots),
                     lambda: kvcache.attention(dual, cache, table, slots), lambda: kvcache.attention(x, cache, table, slots, out=dual)):
            with pytest.raises(NotImplementedError, match="forward-mode"):
                call()
