"""The operators of the key-value cache together, as a serving program uses them: a
layer over steps of prompts and single tokens, on other streams, in graphs, through
the C ABI."""

import math

import pytest

import kv_util as ref
from gpu_util import log, need_gpu

pytestmark = pytest.mark.gpu

HIDDEN, HEADS, KV, D, PAGE = 256, 4, 2, 64, 16


def _layer(torch, seed, window=0):
    from mxfp8_block_scaled_quantize_amd import rotary
    from mxfp8_block_scaled_quantize_amd.attention_layer import MXFP4Attention
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*s):
        return torch.randn(s, generator=g, device="cuda")
    turns, magnitude = rotary.turns(32, scaling="yarn", factor=4.0, trained=512)
    layer = MXFP4Attention(HIDDEN, HEADS, KV, D, turns, magnitude, window=window, device="cuda")
    return layer.load((normal((HEADS + 2 * KV) * D, HIDDEN) * 0.08).bfloat16(), (normal(HIDDEN, HEADS * D) * 0.08).bfloat16()), normal


def _plain_step(torch, layer, x, plan, state):
    """The layer's output in 64 bits: the MXFP4 roundings of the library's quantizer (tested on its own), everything
    between them plain; the keys and values of each request are kept in `state`."""
    from mxfp8_block_scaled_quantize_amd import mxfp4

    def values(t):
        q = mxfp4.quantize(t.contiguous(), packed=True)
        return mxfp4.dequantize(q["q_row"], q["p_row"]).double()
    qkv = (values(x) @ mxfp4.dequantize(layer.qkv, layer.qkv_scales).double().t()).bfloat16().view(-1, HEADS + 2 * KV, D)
    q, k, v = qkv.split((HEADS, KV, KV), 1)
    q, k = (ref.rotate(t, plan.positions, layer.turns, layer.magnitude, False)[0].bfloat16() for t in (q, k))
    out = torch.zeros((x.shape[0], HEADS * D), dtype=torch.float64, device="cuda")
    offsets = plan.offsets.tolist()
    for b in range(len(offsets) - 1):
        i0, i1 = offsets[b], offsets[b + 1]
        if i0 == i1:
            continue
        for name, t in (("k", k), ("v", v)):
            new = values(t[i0:i1].reshape(-1, D).repeat(1, 2)).view(i1 - i0, KV, 2 * D)[..., :D]
            state[b][name] = torch.cat((state[b][name], new))
        kk, vv = state[b]["k"], state[b]["v"]
        at = torch.arange(len(kk) - (i1 - i0), len(kk), device="cuda")[:, None]
        key = torch.arange(len(kk), device="cuda")
        sees = (key <= at) & ((key > at - layer.window) if layer.window else True)
        for h in range(HEADS):
            s = (q[i0:i1, h].double() @ kk[:, h // (HEADS // KV)].t()) * D ** -0.5
            p = torch.softmax(torch.where(sees, s, -math.inf), 1)
            out[i0:i1, h * D:(h + 1) * D] = p @ vv[:, h // (HEADS // KV)]
    return values(out.bfloat16()) @ mxfp4.dequantize(layer.out, layer.out_scales).double().t()


@pytest.mark.parametrize("window", [0, 24])
def test_steps(window):
    """Prompts, then single tokens, then a piece and tokens mixed, then a request that leaves and its pages used again."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    layer, normal = _layer(torch, 1, window)
    n, pages = 3, 40
    cache = kvcache.new(pages, PAGE, KV, D, device="cuda")
    free, left = kvcache.pool(pages, device="cuda")
    table = torch.full((n, 16), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(n, dtype=torch.int32, device="cuda")
    empty = torch.zeros((0, KV, D), dtype=torch.float64, device="cuda")
    state = [{"k": empty, "v": empty} for _ in range(n)]
    for step, counts in enumerate(([37, 5, 80], [1, 1, 1], [1, 0, 1], [20, 1, 1], None, [30, 2, 1])):
        log("step %d: %s" % (step, counts))
        if counts is None:
            finished = torch.tensor([True, False, False], device="cuda")
            lengths, left = kvcache.release(table, lengths, finished, free, left, PAGE)
            state[0] = {"k": empty, "v": empty}
            continue
        rows = sum(counts) + 2      # two padded rows
        x = normal(rows, HIDDEN).bfloat16()
        plan = kvcache.extend(table, lengths, torch.tensor(counts, dtype=torch.int32, device="cuda"), free, left, rows, PAGE)
        lengths, left = plan.lengths, plan.free_count
        got = layer(x, cache, table, plan, max_queries=max(counts))
        want = _plain_step(torch, layer, x, plan, state)
        kept = slice(0, sum(counts))
        # a value that lies next to a border between two codes may round to the other one: the norm, not each element
        assert (got[kept].double() - want[kept]).norm() <= 0.03 * want[kept].norm(), step
        assert lengths.tolist() == [len(s["k"]) for s in state]


def _decode(torch, seed):
    """One decoding step's inputs: a filled cache and a function that runs the operators one after another."""
    from mxfp8_block_scaled_quantize_amd import kvcache, rotary
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, width = 5, 300
    cache = torch.zeros((n * width, KV, PAGE * 68), dtype=torch.uint8, device="cuda")
    table = torch.randperm(n * width, generator=g, device="cuda").to(torch.int32).view(n, width)
    lengths = torch.tensor([4000, 10, 700, 0, 33], dtype=torch.int32, device="cuda")
    kv = torch.randn((n * width * PAGE, KV, D), generator=g, device="cuda").bfloat16()
    kvcache.append(cache, kv, kv.flip(0), torch.arange(n * width * PAGE, dtype=torch.int32, device="cuda"))
    x = torch.randn((n, HEADS + 2 * KV, D), generator=g, device="cuda").bfloat16()
    counts = torch.ones(n, dtype=torch.int32, device="cuda")
    free, left = kvcache.pool(4, device="cuda")
    turns = rotary.turns(D, device="cuda")[0]

    def run(x):
        plan = kvcache.extend(table, lengths, counts, free, left, n, PAGE)
        q, k, v = x.split((HEADS, KV, KV), 1)
        q, k = rotary.rotate(q, k, plan.positions, turns)
        kvcache.append(cache, k, v, plan.slots)
        out, lse = kvcache.attention(q, cache, table, plan.lengths, plan.offsets, max_queries=1, lse=True)
        return out, lse, plan.slots, *kvcache.read(cache, plan.slots, D)
    return run, x, g, (table, lengths, cache)


def test_in_a_graph():
    torch = need_gpu()
    run, x, g, (table, lengths, cache) = _decode(torch, 2)
    want_first = [t.clone() for t in run(x)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(x)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(x)
    for i in range(5):
        log("replay %d" % i)
        x.copy_(torch.randn(x.shape, generator=g, device="cuda").bfloat16())
        if i:
            lengths.copy_(torch.randint(0, 4700, (5,), generator=g, device="cuda", dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        for a, b in zip(got, run(x)):
            assert torch.equal(a, b)
    assert want_first[0].shape == (5, HEADS, D)


def test_two_graphs_share_a_pool():
    """Two captured steps whose workspaces come from one pool, replayed in turn."""
    torch = need_gpu()
    a, xa, _, _ = _decode(torch, 3)
    b, xb, _, _ = _decode(torch, 4)
    want = [[t.clone() for t in f(x)] for f, x in ((a, xa), (b, xb))]
    torch.cuda.synchronize()
    graphs, outs = [], []
    pool = torch.cuda.graph_pool_handle()
    for f, x in ((a, xa), (b, xb)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, pool=pool):
            outs.append(f(x))
        graphs.append(graph)
    for _ in range(3):
        for graph, out, w in zip(graphs, outs, want):
            graph.replay()
            torch.cuda.synchronize()
            # (the other graph may use this one's memory once it is replayed: looked at now)
            for got, x in zip(out, w):
                assert torch.equal(got, x)


def _rotary_step(torch, seed):
    from mxfp8_block_scaled_quantize_amd import rotary
    g = torch.Generator(device="cuda").manual_seed(seed)
    q, k, dq, dk = (torch.randn((9, h, 64), generator=g, device="cuda").bfloat16() for h in (4, 2, 4, 2))
    positions = torch.arange(9, device="cuda", dtype=torch.int32)
    turns = rotary.turns(64, device="cuda")[0]

    def forward(q, k):
        return rotary.rotate(q, k, positions, turns)

    def step(q, k):
        return torch.autograd.grad(forward(q, k), (q, k), (dq, dk))
    return q, k, dq, dk, forward, step


def _capture(torch, step, q, k):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q.clone().detach().requires_grad_(), k.clone().detach().requires_grad_())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = step(q, k)
    return graph, grads


def test_rotary_gradients_in_a_graph():
    torch = need_gpu()
    q, k, dq, dk, _, step = _rotary_step(torch, 1)
    held_q, held_k = q.clone().requires_grad_(), k.clone().requires_grad_()
    graph, (gq, gk) = _capture(torch, step, held_q, held_k)
    for i in range(4):
        log("replay %d" % i)
        dq.copy_(torch.randn_like(dq))
        dk.copy_(torch.randn_like(dk))
        graph.replay()
        torch.cuda.synchronize()
        wq, wk = step(q.clone().requires_grad_(), k.clone().requires_grad_())
        assert torch.equal(gq, wq) and torch.equal(gk, wk)


def test_rotary_gradients_are_not_captured_beside_a_living_graph():
    """A graph of the same leaves, made on another stream, would end the process at the capture's end: refused."""
    torch = need_gpu()
    q, k, dq, dk, forward, step = _rotary_step(torch, 2)
    held_q, held_k = q.clone().requires_grad_(), k.clone().requires_grad_()
    alive = forward(held_q, held_k)
    with pytest.raises(RuntimeError, match="cannot be captured while a graph"):
        _capture(torch, step, held_q, held_k)
    torch.cuda.synchronize()
    # the forward pass alone can be captured, and the other graph still has its gradients
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = forward(held_q, held_k)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[0], alive[0]) and torch.equal(out[1], alive[1])
    want = step(q.clone().requires_grad_(), k.clone().requires_grad_())
    for a, b in zip(torch.autograd.grad(alive, (held_q, held_k), (dq, dk)), want):
        assert torch.equal(a, b)
    # without it the pass can be captured
    del alive, out
    graph, grads = _capture(torch, step, held_q, held_k)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(grads, want):
        assert torch.equal(a, b)


def test_on_another_stream():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache, rotary
    run, x, _, (table, lengths, cache) = _decode(torch, 5)
    want = [t.clone() for t in run(x)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = run(x)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # stream arguments, a torch stream and a raw handle
    q = x[:, :HEADS].contiguous()
    positions = torch.arange(5, device="cuda", dtype=torch.int32)
    turns = rotary.turns(D, device="cuda")[0]
    free, left = kvcache.pool(4, device="cuda")
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        a = rotary.rotate(q, None, positions, turns, stream=stream)
        b = kvcache.attention(q, cache, table, lengths, stream=stream)
        c = kvcache.read(cache, positions, D, stream=stream)
        plan = kvcache.extend(table.clone(), lengths, positions, free, left, 20, PAGE, stream=stream)
        side.synchronize()
        assert torch.equal(a, rotary.rotate(q, None, positions, turns))
        assert torch.equal(b, kvcache.attention(q, cache, table, lengths))
        assert all(torch.equal(u, v) for u, v in zip(c, kvcache.read(cache, positions, D)))
        assert torch.equal(plan.offsets, torch.tensor([0, 0, 1, 3, 6, 10], dtype=torch.int32, device="cuda"))
        twin = cache.clone()
        torch.cuda.synchronize()
        kvcache.append(twin, c[0], c[1], positions + 100, stream=stream)
        kvcache.release(table.clone(), lengths, lengths > 0, free.clone(), left, PAGE, stream=stream)
        side.synchronize()
        kvcache.append(cache, c[0], c[1], positions + 100)
        assert torch.equal(twin, cache)


@pytest.mark.parametrize("side", [False, True])
def test_c_mirror(side):
    """The functions that mirror the C ABI, on tensors of the caller's own."""
    torch = need_gpu()
    import mxfp8_block_scaled_quantize_amd as mx
    from mxfp8_block_scaled_quantize_amd import kvcache, rotary
    log("C mirror of the key-value cache, side stream %s" % side)
    _, x, _, (table, lengths, cache) = _decode(torch, 6)
    pages, width, n = cache.shape[0], table.shape[1], 5
    q, k, v = x.split((HEADS, KV, KV), 1)
    counts = torch.ones(n, dtype=torch.int32, device="cuda")
    free, left = kvcache.pool(pages, device="cuda")
    turns = rotary.turns(D, device="cuda")[0]
    twin = cache.clone()
    plan = kvcache.extend(table, lengths, counts, free, left, n, PAGE)
    wq, wk = rotary.rotate(q, k, plan.positions, turns)
    kvcache.append(cache, wk, v, plan.slots)
    want, want_lse = kvcache.attention(wq, cache, table, plan.lengths, lse=True)
    i32 = dict(dtype=torch.int32, device="cuda")
    stream = torch.cuda.Stream() if side else None
    raw = stream.cuda_stream if side else None
    offsets, out_lengths, slots, positions, out_left = (torch.full((m,), 77, **i32) for m in (n + 1, n, n, n, 1))
    gq, gk = torch.zeros_like(wq), torch.zeros_like(wk)
    need = kvcache.kv_attention_workspace_bytes(n, HEADS, KV, D, n, width, PAGE, 0, 1, 0)
    assert need > 0
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(want), torch.zeros_like(want_lse)
    rk, rv = torch.zeros_like(wk), torch.zeros_like(wk)
    torch.cuda.synchronize()
    kvcache.kv_extend(table, width, width, lengths, counts, n, free, left, pages, PAGE, n, offsets, out_lengths, slots, positions,
                      out_left, stream=stream)
    rotary.rotary_rotate(q, q.stride(0), q.stride(1), HEADS, k, k.stride(0), k.stride(1), KV, rotary.ROTARY_BF16, n, D, D // 2, positions,
                         turns, 1.0, 0, gq, gk, stream=stream)
    kvcache.kv_append(twin, pages, PAGE, KV, D, gk, KV * D, D, v, v.stride(0), v.stride(1), slots, n, stream=raw)
    kvcache.kv_attention(gq, HEADS * D, D, n, HEADS, twin, pages, PAGE, KV, D, table, width, width, out_lengths, None, n, 1, D ** -0.5, 0,
                         out, lse, work, need, stream=stream)
    kvcache.kv_read(twin, pages, PAGE, KV, D, slots, n, rk, rv, stream=stream)
    torch.cuda.synchronize()
    for a, b in ((offsets, plan.offsets), (out_lengths, plan.lengths), (slots, plan.slots), (positions, plan.positions), (out_left, plan.free_count),
                 (gq, wq), (gk, wk), (twin, cache), (out, want), (lse, want_lse), (rk, kvcache.read(cache, slots, D)[0])):
        assert torch.equal(a, b)
    finished = torch.tensor([1, 0, 1, 0, 0], dtype=torch.uint8, device="cuda")
    t2, f2 = table.clone(), free.clone()
    torch.cuda.synchronize()
    kvcache.kv_release(table, width, width, out_lengths, finished, n, free, out_left, pages, PAGE, lengths, left, stream=stream)
    torch.cuda.synchronize()
    w_lengths, w_left = kvcache.release(t2, out_lengths, finished.bool(), f2, out_left, PAGE)
    for a, b in ((lengths, w_lengths), (left, w_left), (table, t2), (free, f2)):
        assert torch.equal(a, b)
    with pytest.raises(mx.MXFP8Error, match="kv_attention"):
        kvcache.kv_attention(gq, HEADS * D, D, n, HEADS, twin, pages, PAGE, KV, D, table, width, width, out_lengths, None, n, 1, 0.0, 0, out)


def test_no_rows_and_no_free_pages():
    """A step without rows, and one whose requests get no page: lengths and cache stay as they were."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import kvcache
    layer, normal = _layer(torch, 3, 0)
    cache = kvcache.new(4, PAGE, KV, D, device="cuda")
    free, _ = kvcache.pool(4, device="cuda")
    none = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lengths = torch.zeros(2, dtype=torch.int32, device="cuda")
    for rows, counts in ((0, [0, 0]), (9, [3, 5])):
        log("%d rows" % rows)
        plan = kvcache.extend(table, lengths, torch.tensor(counts, dtype=torch.int32, device="cuda"), free, none, rows, PAGE)
        assert plan.lengths.tolist() == [0, 0] and bool((plan.slots == -1).all()) and plan.free_count.tolist() == [0]
        assert layer(normal(rows, HIDDEN).bfloat16(), cache, table, plan).shape == (rows, HIDDEN)
        assert not bool(cache.any()) and bool((table == -1).all())
