"""Options without a truth value are an error of their own (no GPU needed)."""

import numpy as np
import pytest
import torch

from mxfp8_block_scaled_quantize_amd import mxfp4


@pytest.mark.parametrize("value", [np.array([1, 2]), torch.tensor([True, False])], ids=["array", "tensor"])
def test_no_truth_value(value):
    x = torch.zeros((32, 128), dtype=torch.bfloat16)
    codes, words = torch.zeros((32, 64), dtype=torch.uint8), torch.zeros((1, 32), dtype=torch.int32)
    for name in ("rowwise", "colwise", "packed"):
        with pytest.raises((ValueError, RuntimeError), match="ambiguous"):
            mxfp4.quantize(x, **{name: value})
    for name in ("accumulate", "swiglu"):
        with pytest.raises((ValueError, RuntimeError), match="ambiguous"):
            mxfp4.gemm(codes, words, codes, words, **{name: value})
        with pytest.raises((ValueError, RuntimeError), match="ambiguous"):
            mxfp4.grouped_gemm(codes, words, codes.view(1, 32, 64), words, words[0], **{name: value})
