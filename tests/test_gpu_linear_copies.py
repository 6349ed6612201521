"""MXFP8Linear's kept weight copies on several streams and in captured graphs."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu

K, N = 1024, 2048


def _layer(torch, seed):
    from mxfp8_block_scaled_quantize_amd.linear import MXFP8Linear
    layer = MXFP8Linear(K, N, device="cuda")
    _set(torch, layer, seed)
    return layer


def _set(torch, layer, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    with torch.no_grad():
        layer.weight.copy_(torch.randn((N, K), generator=g, device="cuda"))


def _want(torch, layer, x):
    """The layer's product of separately made copies."""
    from mxfp8_block_scaled_quantize_amd.linear import mxfp8_linear_inference
    return mxfp8_linear_inference(x, layer.weight.detach())


def _x(torch, seed):
    return torch.randn((256, K), generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").bfloat16()


def test_streams():
    torch = need_gpu()
    log("MXFP8Linear on streams")
    layer, x = _layer(torch, 1), _x(torch, 2)
    sides = [torch.cuda.Stream() for _ in range(3)]
    with torch.no_grad():
        for seed in range(6):
            _set(torch, layer, seed)
            for s in sides:
                s.wait_stream(torch.cuda.current_stream())
            got = []
            for s in sides:              # the first one quantizes, the others wait for its copies
                with torch.cuda.stream(s):
                    got.append(layer(x))
            assert layer._wq_stream == sides[0].cuda_stream
            for s in sides:
                torch.cuda.current_stream().wait_stream(s)
            want = _want(torch, layer, x)
            assert all(torch.equal(y, want) for y in got)


def test_first_call_in_a_capture_and_later_weights():
    torch = need_gpu()
    log("MXFP8Linear captured")
    other, layer, x = _layer(torch, 0), _layer(torch, 1), _x(torch, 2)
    with torch.no_grad():
        other(x)                          # warm-up of another layer: this one's first call is the captured one
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x)
        assert layer._wq is None
        assert torch.equal(layer(x), _want(torch, layer, x))       # eager, before any replay
        for seed in range(3):
            _set(torch, layer, seed)
            junk = [torch.full((N, K), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, _want(torch, layer, x))
            assert torch.equal(layer(x), out)
            del junk


def test_kept_copies_are_not_captured():
    torch = need_gpu()
    log("MXFP8Linear with copies, captured")
    layer, x = _layer(torch, 1), _x(torch, 2)
    with torch.no_grad():
        layer(x)                          # copies are there
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = layer(x)
        for seed in range(3):
            _set(torch, layer, seed)
            layer(x)                      # and are made anew
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, _want(torch, layer, x))
