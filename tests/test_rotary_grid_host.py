"""Rotary positions of as many elements as a launch's threads turn: a thread takes 16 bytes
of each of two runs and of up to eight heads, so the limit is that of the threads."""

from mxfp8_block_scaled_quantize_amd import rotary

P = 0x10000   # fake, aligned "device" addresses: never dereferenced, a missing one is refused behind the limits
NULL, LIMIT = 1, 7


def _status(tokens, heads, d, pairs, dtype=rotary.ROTARY_BF16, q_stride=None):
    f = rotary._functions()["rotary_rotate"]
    return f(P, heads * d if q_stride is None else q_stride, d, heads, P, 0, 0, 0, dtype, tokens, d, pairs, None, P, 1.0, 0, P, P, None)


def test_limits():
    # 2^20 tokens of 40 heads of 128: 5.4e9 elements, 4.2e7 threads
    assert _status(1 << 20, 40, 128, 64) == NULL
    assert _status(1 << 24, 40, 128, 64) == NULL
    assert _status(1 << 24, 40, 128, 64, rotary.ROTARY_FP32) == NULL
    # 2^28 tokens of 8 runs and 5 groups of heads: more threads than a launch has
    assert _status(1 << 28, 40, 128, 64) == LIMIT
    # an odd stride: a pair and thread each
    assert _status(1 << 22, 40, 128, 64, q_stride=40 * 128 + 1) == NULL
    assert _status(1 << 24, 40, 128, 64, q_stride=40 * 128 + 1) == LIMIT
    assert _status(1 << 30, 6, 64, 32) == LIMIT and _status((1 << 40) - 1, 1, 64, 32, q_stride=0) == LIMIT
    assert _status((1 << 63) - 1, 1, 64, 32, q_stride=0) == LIMIT
