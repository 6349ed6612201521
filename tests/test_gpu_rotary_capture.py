"""Captured gradients of rotary positions whose queries and keys are made of leaves by
other operators: beside a living graph of these leaves, made on another stream, the pass
would end the process and is refused; without it, or where it does not lead to the
leaves, it is captured."""

import pytest

from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu


def _step(torch, seed):
    from mxfp8_block_scaled_quantize_amd import rotary
    g = torch.Generator(device="cuda").manual_seed(seed)
    leaf = torch.randn((9, 6 * 64), generator=g, device="cuda").bfloat16()
    dq, dk = (torch.randn((9, h, 64), generator=g, device="cuda").bfloat16() for h in (4, 2))
    positions = torch.arange(9, device="cuda", dtype=torch.int32)
    turns = rotary.turns(64, device="cuda")[0]

    def split(leaf):
        return (leaf * 1.5).view(9, 6, 64).split((4, 2), 1)

    def forward(leaf):
        return rotary.rotate(*split(leaf), positions, turns)

    def step(leaf):
        return torch.autograd.grad(forward(leaf), (leaf,), (dq, dk))

    def inner(leaf):
        q, k = split(leaf)
        return torch.autograd.grad(rotary.rotate(q, k, positions, turns), (q, k), (dq, dk))

    def whole(leaf):
        leaf.grad = None
        torch.autograd.backward(forward(leaf), (dq, dk))
        return (leaf.grad,)
    return leaf, dq, dk, forward, {"grad": step, "inner": inner, "backward": whole}


def _capture(torch, step, leaf):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(leaf.detach().clone().requires_grad_())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(leaf)
    return graph, out


@pytest.mark.parametrize("kind", ["grad", "inner", "backward"])
def test_without_a_living_graph(kind):
    torch = need_gpu()
    log(kind)
    leaf, dq, dk, _, steps = _step(torch, 1)
    held = leaf.clone().requires_grad_()
    graph, out = _capture(torch, steps[kind], held)
    for i in range(3):
        dq.copy_(torch.randn_like(dq))
        dk.copy_(torch.randn_like(dk))
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, steps[kind](leaf.clone().requires_grad_())):
            assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["grad", "backward"])
def test_beside_a_living_graph(kind):
    torch = need_gpu()
    log(kind)
    leaf, dq, dk, forward, steps = _step(torch, 2)
    held = leaf.clone().requires_grad_()
    alive = forward(held)
    with pytest.raises(RuntimeError, match="cannot be captured while a graph"):
        _capture(torch, steps[kind], held)
    torch.cuda.synchronize()
    want = steps["grad"](leaf.clone().requires_grad_())
    # the other graph still has its gradients; without it the pass can be captured
    assert torch.equal(torch.autograd.grad(alive, (held,), (dq, dk))[0], want[0])
    del alive
    graph, out = _capture(torch, steps[kind], held)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], want[0])


def test_a_pass_that_ends_before_the_leaves():
    torch = need_gpu()
    leaf, dq, dk, forward, steps = _step(torch, 3)
    held = leaf.clone().requires_grad_()
    alive = forward(held)
    graph, out = _capture(torch, steps["inner"], held)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, steps["inner"](leaf.clone().requires_grad_())):
        assert torch.equal(a, b)
    assert alive[0].requires_grad
