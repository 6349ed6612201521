"""MXFP4Linear's weight copies on several streams and in captured graphs."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu

K, N = 1024, 2048


def _layer(torch, seed):
    from mxfp8_block_scaled_quantize_amd.mxfp4_linear import MXFP4Linear
    layer = MXFP4Linear(K, N, device="cuda")
    _set(torch, layer, seed)
    return layer


def _set(torch, layer, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    layer.weight.data.copy_(torch.randn((N, K), generator=g, device="cuda"))


def _want(torch, layer, x):
    """The layer's product of separately made copies."""
    from mxfp8_block_scaled_quantize_amd import mxfp4
    q, w = mxfp4.quantize(x, packed=True), mxfp4.quantize(layer.weight.detach(), packed=True)
    return mxfp4.gemm(q["q_row"], q["p_row"], w["q_row"], w["p_row"])


def _x(torch, seed):
    return torch.randn((256, K), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


@pytest.mark.parametrize("frozen", [False, True])
def test_streams(frozen):
    torch = need_gpu()
    log("MXFP4Linear on streams, frozen=%s" % frozen)
    layer, x = _layer(torch, 1), _x(torch, 2)
    sides = [torch.cuda.Stream() for _ in range(3)]
    with torch.no_grad():
        for seed in range(4):
            _set(torch, layer, seed)
            if frozen:
                layer.freeze_weight()
            for s in sides:
                s.wait_stream(torch.cuda.current_stream())
            got = []
            for s in sides:              # each on its own, none waits for another
                with torch.cuda.stream(s):
                    got.append(layer(x))
            for s in sides:
                torch.cuda.current_stream().wait_stream(s)
            want = _want(torch, layer, x)
            assert all(torch.equal(y, want) for y in got)
            if frozen:
                layer.thaw_weight()


def test_first_call_in_a_capture_and_later_weights():
    torch = need_gpu()
    log("MXFP4Linear captured")
    other, layer, x = _layer(torch, 0), _layer(torch, 1), _x(torch, 2)
    with torch.no_grad():
        other(x)                          # warm-up of another layer: this one's first call is the captured one
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x)
        assert torch.equal(layer(x), _want(torch, layer, x))       # eager, before any replay
        for seed in range(3):
            _set(torch, layer, seed)
            junk = [torch.full((N, K // 2), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, _want(torch, layer, x))
            assert torch.equal(layer(x), out)
            del junk


def test_frozen_copies_in_a_graph():
    torch = need_gpu()
    log("MXFP4Linear frozen, captured")
    layer, x = _layer(torch, 1).freeze_weight(), _x(torch, 2)
    with torch.no_grad():
        layer(x)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x)
        for seed in range(3):
            _set(torch, layer, seed)
            layer.freeze_weight()           # in place: the graph follows
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, _want(torch, layer, x)) and torch.equal(layer(x), out)


def test_freezing_is_refused_in_a_capture():
    torch = need_gpu()
    log("MXFP4Linear frozen in a capture")
    layer, x = _layer(torch, 1), _x(torch, 2)
    graph = torch.cuda.CUDAGraph()
    with torch.no_grad(), torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            layer.freeze_weight()
        out = layer(x)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _want(torch, layer, x))


def test_training_step_with_master_weights():
    torch = need_gpu()
    log("MXFP4Linear with master weights")
    layer, x = _layer(torch, 1), _x(torch, 2)
    dy = torch.randn((256, N), device="cuda").bfloat16()
    master = layer.weight.detach().float()
    for _ in range(3):
        y = layer(x)
        assert torch.equal(y.detach(), _want(torch, layer, x))
        y.backward(dy)
        master -= 0.5 * layer.weight.grad.float() / layer.weight.grad.float().abs().max()
        layer.weight.data.copy_(master)     # leaves the weight's version as it is
        layer.weight.grad = None
