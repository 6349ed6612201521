"""What stands in front of a window does not matter either: bytes of NaN in the places
that the tile's first query no longer sees, up to the next 32 or 64 keys, change no bit."""

import pytest

from gpu_util import log, need_gpu
from test_gpu_kv_attention import Case

pytestmark = pytest.mark.gpu


def _fill_front(c, byte, ends):
    """Every byte of the keys and values in front of key ends[b] of sequence b."""
    page, d = c.page, c.d
    half, few = page * d // 2, page * d // 32
    for b, end in enumerate(ends):
        for j in range(-(-end // page)):
            n = min(page, end - j * page)
            r = c.cache[int(c.table[b, j])]
            r[:, :half].view(-1, page, d // 2)[:, :n] = byte
            v = r[:, half:2 * half].view(-1, page // 4, d // 8, 4, 4)
            for i in range(n):
                v[:, i // 4, :, i % 4] = byte
            r[:, 2 * half:2 * half + few].view(-1, page, d // 32)[:, :n] = byte
            r[:, 2 * half + few:].view(-1, d // 32, page)[..., :n] = byte


@pytest.mark.parametrize("byte", [0xFF, 0x7F])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("most", [1, 12, 90])
def test_bytes_in_front_of_the_window(byte, d, page, most):
    torch = need_gpu()
    window = 47
    lengths, queries = [200, 333, 100, 7000, 59], [1, 3, 90, 12, 1]
    log("byte %#x D=%d page=%d most=%d" % (byte, d, page, most))
    a, b = (Case(lengths, queries, 4, 2, d, page, seed=4) for _ in range(2))
    # the first key that a sequence's first query sees
    _fill_front(b, byte, [max(0, n - q + 1 - window) for n, q in zip(lengths, queries)])
    assert not torch.equal(a.cache, b.cache)
    want, got = a.run(max_queries=most, window=window), b.run(max_queries=most, window=window)
    assert bool(torch.isfinite(want[0]).all())
    for x, y in zip(got, want):
        assert torch.equal(x, y)
