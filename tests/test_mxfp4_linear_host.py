"""MXFP4Linear's weight copies, host logic alone: the quantizer and the product
are stand-ins, so that no GPU is needed.  A call uses the weight's value of that
moment, unless the weight has been frozen."""

import copy
import pickle

import pytest
import torch

import mxfp8_block_scaled_quantize_amd.mxfp4_linear as lin

K, N = 128, 256


@pytest.fixture
def calls(monkeypatch):
    """Shapes that were quantized, with the copies asked for."""
    made = []

    def quantize(t, rowwise=True, colwise=False, packed=False):
        made.append((tuple(t.shape), rowwise, colwise))
        q = {}
        if rowwise:
            q["q_row"], q["p_row"] = t.float(), t.float()
        if colwise:
            q["q_colT"], q["p_colT"] = t.t().float(), t.t().float()
        return q

    monkeypatch.setattr(lin, "quantize", quantize)
    monkeypatch.setattr(lin, "gemm", lambda a, ap, b, bp: (a @ b.t()).bfloat16())
    return made


def _weights(calls):
    return [c for c in calls if c[0] == (N, K)]


def _input(grad=False):
    return torch.randn((128, K)).bfloat16().requires_grad_(grad)


def _expect(layer, x, w=None):
    return (x.float() @ (layer.weight if w is None else w).detach().float().t()).bfloat16()


def _writes(layer):
    """Ways to change the weight, most of them without a trace in its version."""
    new = torch.randn((N, K)).bfloat16()

    def in_place():
        with torch.no_grad():
            layer.weight.copy_(new)

    def through_data():
        layer.weight.data.copy_(new)

    def data_replaced():
        layer.weight.data = new.clone()

    def parameter_replaced():
        layer.weight = torch.nn.Parameter(new.clone())

    def storage_written():
        torch.frombuffer(layer.weight.data.view(torch.int16).numpy(), dtype=torch.int16).copy_(new.view(torch.int16).flatten())
    return {f.__name__: f for f in (in_place, through_data, data_replaced, parameter_replaced, storage_written)}


WRITES = ["in_place", "through_data", "data_replaced", "parameter_replaced", "storage_written"]


@pytest.mark.parametrize("write", WRITES)
@pytest.mark.parametrize("train", [False, True])
def test_every_write_is_seen(calls, write, train):
    layer = lin.MXFP4Linear(K, N)
    x = _input(train)
    with torch.set_grad_enabled(train):
        assert torch.equal(layer(x), _expect(layer, x))
        _writes(layer)[write]()
        y = layer(x)
        assert torch.equal(y, _expect(layer, x))
        if train:
            y.backward(torch.ones_like(y))
            assert torch.equal(x.grad, (torch.ones(128, N) @ layer.weight.detach().float()).bfloat16())


def test_only_the_copies_that_are_read(calls):
    layer = lin.MXFP4Linear(K, N)
    with torch.no_grad():
        layer(_input())
    layer(_input())                    # the weight's gradient alone
    layer(_input(True))
    layer.weight.requires_grad_(False)
    layer(_input(True))
    assert _weights(calls) == [((N, K), True, c) for c in (False, False, True, True)]


def test_frozen_weight(calls):
    layer = lin.MXFP4Linear(K, N)
    assert layer.freeze_weight() is layer
    was = layer.weight.detach().clone()
    del calls[:]
    x = _input()
    with torch.no_grad():
        assert torch.equal(layer(x), _expect(layer, x))
        _writes(layer)["through_data"]()
        assert torch.equal(layer(x), _expect(layer, x, was))     # as documented
    assert not _weights(calls)
    y = layer(_input(True))             # a weight that needs a gradient is taken as it is
    assert _weights(calls) == [((N, K), True, True)] and y.requires_grad
    kept = layer._wq
    layer.freeze_weight()               # in place, and the same tensors
    assert layer._wq[0] is kept[0] and layer._wq[1] is kept[1]
    with torch.no_grad():
        assert torch.equal(layer(x), _expect(layer, x))
        layer.thaw_weight()
        _writes(layer)["through_data"]()
        assert torch.equal(layer(x), _expect(layer, x))


def test_frozen_weight_and_the_gradient_of_the_input(calls):
    layer = lin.MXFP4Linear(K, N)
    layer.weight.requires_grad_(False)
    for colwise, quantized in ((False, 1), (True, 0)):
        layer.freeze_weight(colwise=colwise)
        del calls[:]
        x = _input(True)
        layer(x).backward(torch.ones((128, N), dtype=torch.bfloat16))
        assert len(_weights(calls)) == quantized
        assert torch.equal(x.grad, (torch.ones(128, N) @ layer.weight.float()).bfloat16())
    layer.freeze_weight()               # keeps the transposed copy
    assert layer._wq[2] is not None


@pytest.mark.parametrize("write", ["parameter_replaced", "state_dict", "module_moved"])
def test_what_ends_it(calls, write):
    layer = lin.MXFP4Linear(K, N).freeze_weight()
    if write == "state_dict":
        layer.load_state_dict({"weight": torch.randn((N, K)).bfloat16()})
    elif write == "module_moved":
        layer.to("cpu")
        layer.weight.data.mul_(2)
    else:
        _writes(layer)[write]()
    x = _input()
    with torch.no_grad():
        assert torch.equal(layer(x), _expect(layer, x))
    assert [n for n, _ in layer.named_parameters()] == ["weight"] and list(layer.state_dict()) == ["weight"]


def test_copies_of_a_frozen_layer(calls):
    layer = lin.MXFP4Linear(K, N).freeze_weight()
    for other in (copy.deepcopy(layer), pickle.loads(pickle.dumps(layer))):
        del calls[:]
        x = _input()
        with torch.no_grad():
            assert torch.equal(other(x), _expect(layer, x)) and not _weights(calls)
            other.weight = torch.nn.Parameter(-other.weight.detach())
            assert torch.equal(other(x), _expect(other, x))
            assert torch.equal(layer(x), _expect(layer, x))


def test_frozen_in_inference_mode(calls):
    layer = lin.MXFP4Linear(K, N)
    layer.weight.requires_grad_(False)
    with torch.inference_mode():
        layer.freeze_weight(colwise=True)
        layer(_input())
    x = _input(True)
    layer(x).backward(torch.ones((128, N), dtype=torch.bfloat16))   # the copies can be saved for backward
    assert x.grad is not None
