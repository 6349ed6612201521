"""Products that no kernel's grid can hold are refused (host checks; the
addresses are never used)."""

import pytest

import mxfp8_block_scaled_quantize_amd as mx
from mxfp8_block_scaled_quantize_amd import mxfp4

P = 0x10000
LIMIT = 7


@pytest.mark.parametrize("N", [288, 512])
def test_too_many_tiles(N):
    M = (1 << 31) - 1
    with pytest.raises(mx.MXFP8Error) as e:
        mxfp4.mxfp4_gemm(P, P, P, P, P, N, M, N, 128, 0, stream=0)
    assert e.value.status == LIMIT
    with pytest.raises(mx.MXFP8Error) as e:
        mxfp4.mxfp4_grouped_gemm(P, P, P, P, P, 2, P, N, M, N, 128, 0, stream=0)
    assert e.value.status == LIMIT
