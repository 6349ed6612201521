"""MXFP8Linear's kept weight copies, host logic alone (the quantizer is a
stand-in): what makes them anew."""

import copy
import pickle

import pytest
import torch

import mxfp8_block_scaled_quantize_amd.linear as lin


@pytest.fixture
def made(monkeypatch):
    """Values of the weights that were quantized."""
    values = []

    def quantize(t, **kw):
        values.append(float(t[0, 0]))
        c = t.clone()
        return {"q_row": c, "p_row": c, "q_colT": c, "p_colT": c}
    monkeypatch.setattr(lin, "quantize", quantize)
    return values


def _layer(value):
    layer = lin.MXFP8Linear(128, 128)
    with torch.no_grad():
        layer.weight.fill_(value)
    return layer


def test_another_parameter_on_the_same_storage(made):
    layer = _layer(1.0)
    layer.quantized_weight()
    old = layer.weight
    new = torch.nn.Parameter(old.data)
    with torch.no_grad():
        while new._version < old._version:
            new.fill_(2.0)
    assert (new.data_ptr(), new._version) == (old.data_ptr(), old._version)
    layer.weight = new
    assert float(layer.quantized_weight()[0][0, 0]) == 2.0


def test_another_storage_at_the_same_address(made):
    layer = _layer(1.0)
    layer.quantized_weight()
    address = layer.weight.data_ptr()
    layer.weight.data = torch.zeros((128, 128), dtype=torch.bfloat16)
    fresh = [torch.full((128, 128), 3.0, dtype=torch.bfloat16) for _ in range(64)]
    assert address not in [t.data_ptr() for t in fresh]     # the copies' weight is still there
    for t in fresh:
        layer.weight.data = t
        assert float(layer.quantized_weight()[0][0, 0]) == 3.0


def test_forgotten(made):
    layer = _layer(1.0)
    layer.quantized_weight()
    layer.weight.data.fill_(2.0)
    layer.forget_quantized_weight()
    assert float(layer.quantized_weight()[0][0, 0]) == 2.0
    layer.to("cpu")
    assert layer._wq is None and layer._wq_key is None


def test_copies_of_the_layer(made):
    layer = _layer(1.0)
    layer.quantized_weight()
    for other in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        other.weight.data.fill_(5.0)
        assert float(other.quantized_weight()[0][0, 0]) == 5.0
        assert float(layer.quantized_weight()[0][0, 0]) == 1.0


def test_inference_mode(made):
    layer = _layer(1.0)
    with torch.inference_mode():
        q = layer.quantized_weight()
    assert not any(t.is_inference() for t in q) and layer.quantized_weight() is q
    with torch.inference_mode():
        layer = lin.MXFP8Linear(128, 128)
        assert layer.weight.is_inference()
        for value in (1.0, 2.0):
            layer.weight.fill_(value)
            assert float(layer.quantized_weight()[0][0, 0]) == value
