"""The workspace of the attention, which the sizes of a call give on the host: tables far
wider than the sequences in them (as wide as the longest request a program admits) do not
make it large."""

import pytest

from mxfp8_block_scaled_quantize_amd import kvcache

MOST = 80 << 20


def _bytes(tokens, heads, kv_heads, d, sequences, capacity, queries, page=16, ragged=1, window=0):
    return kvcache.kv_attention_workspace_bytes(tokens, heads, kv_heads, d, sequences, capacity // page, page, ragged, queries, window)


@pytest.mark.parametrize("capacity", [4608, 32768, 131072, 1 << 20, 1 << 24])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("tokens,heads,kv_heads,sequences,queries", [
    (8800, 32, 8, 4, 4096), (8192, 32, 8, 4, 4096), (16384, 64, 8, 1, 16384), (1 << 20, 64, 8, 1, 1 << 20), (2048, 32, 8, 64, 2048),
    (512, 32, 8, 512, 1), (4096, 128, 8, 4096, 1), (100000, 32, 8, 4, 1), (500, 32, 8, 1, 500), (1, 8, 1, 1, 1), (65535, 1, 1, 65535, 1)])
def test_it_is_bounded(capacity, d, tokens, heads, kv_heads, sequences, queries):
    assert _bytes(tokens, heads, kv_heads, d, sequences, capacity, queries) <= MOST


@pytest.mark.parametrize("d", [64, 128, 256])
def test_parts_that_fill_the_chip_fit(d):
    """The bound is no less than what the parts take that give every compute unit its workgroups."""
    for tokens, queries, parts in ((8 * 128, 128, 8), (16 * 128, 128, 4), (32 * 128, 128, 2)):   # 512 tiles of 128 rows with 8 heads
        got = _bytes(tokens, 8, 8, d, tokens // 128, 16384, queries)
        assert got // (tokens * 8 * (d + 2) * 4) == parts
    assert _bytes(1, 32, 8, d, 1, 131072, 1, ragged=0) // (32 * (d + 2) * 4) == 32


def test_rows_without_room_for_parts():
    """More rows than two parts have room for: one part, whatever the table's width or the hint."""
    for capacity in (1 << 20, 1 << 24):
        for queries in (1, 1 << 24):
            assert _bytes(1 << 24, 1, 1, 64, 1, capacity, queries) == 0
        assert _bytes(1 << 23, 1, 1, 64, 1 << 23, capacity, 1, ragged=0) == 0
