"""moe.route's order of experts where their choices lie within the rounding of
32 bits: it is the order of the exact scores (ties: lowest index)."""

import numpy as np
import pytest

from gpu_util import log, need_gpu, to_host

pytestmark = pytest.mark.gpu


def _order(x, top_k, scores, bias, groups, top_groups, group_top):
    """Expert ids in 64 bits, by stable sorts."""
    x = x.astype(np.float64)
    if scores == "softmax":
        s = np.exp(x - x.max(1, keepdims=True))
        s /= s.sum(1, keepdims=True)
    else:
        s = 1 / (1 + np.exp(-x))
    v = s if bias is None else s + bias.astype(np.float64)
    if groups > 1:
        inside = -np.sort(-v.reshape(len(v), groups, -1), axis=2)
        best = inside[:, :, :group_top].sum(2)
        keep = np.argsort(-best, axis=1, kind="stable")[:, :top_groups]
        open_ = np.zeros_like(best, dtype=bool)
        np.put_along_axis(open_, keep, True, 1)
        # closed experts behind every open one, whatever its value
        order = np.argsort(-v, axis=1, kind="stable")
        shut = ~np.take_along_axis(np.repeat(open_, v.shape[1] // groups, 1), order, 1)
        order = np.take_along_axis(order, np.argsort(shut, axis=1, kind="stable"), 1)
        return order[:, :top_k]
    return np.argsort(-v, axis=1, kind="stable")[:, :top_k]


# few rows (a wave each) and many, every number of experts a lane holds, groups
# that end with lanes (1, 2, 4, 8, 16 of them) and groups that do not
SHAPES = [(400, 64, 8, 8, 3), (400, 256, 8, 8, 4), (400, 256, 8, 4, 2), (400, 192, 6, 3, 2), (400, 500, 8, 4, 2),
          (400, 1000, 12, 8, 3), (3000, 40, 12, 8, 3), (3000, 64, 9, 16, 5), (3000, 128, 8, 8, 4), (3000, 128, 8, 1, 1),
          (3000, 128, 4, 2, 1), (3000, 256, 8, 32, 9), (3000, 384, 8, 8, 3), (3000, 384, 8, 1, 1), (3000, 640, 10, 10, 4),
          (3000, 96, 1, 6, 1)]


@pytest.mark.parametrize("shape", SHAPES, ids=["%dx%d_k%d_g%d_%d" % s for s in SHAPES])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [1.0, 2.0 ** -10, 2.0 ** -17])
def test_order_is_that_of_the_exact_scores(shape, scores, spread):
    """The smaller the logits' spread, the more choices lie within the rounding:
    of a few rows in a thousand, of most, of all."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe

    T, E, K, groups, top_groups = shape
    log("order %s %s spread=%g" % (shape, scores, spread))
    rng = np.random.default_rng(E + K)
    x = (rng.standard_normal((T, E)) * spread).astype(np.float32)
    # the choices spread like the scores do
    unit = spread if scores == "sigmoid" else spread / E
    bias = (rng.standard_normal(E) * 0.25 * unit).astype(np.float32)
    for b in (bias, None):
        for group_top in (1, 2):
            kw = dict(groups=groups, top_groups=top_groups, group_top=group_top)
            want = _order(x, K, scores, b, **kw)
            w, ids = moe.route(torch.from_numpy(x).cuda(), K, scores=scores,
                               bias=None if b is None else torch.from_numpy(b).cuda(), **kw)
            got = to_host(ids).view(np.int32)
            assert np.array_equal(got, want), (b is not None, group_top, np.flatnonzero((got != want).any(1))[:8])
            assert torch.isfinite(w).all()


@pytest.mark.parametrize("low", [float("-inf"), float(np.finfo(np.float32).min)])
@pytest.mark.parametrize("E,groups", [(64, 8), (128, 8), (60, 6)])
@pytest.mark.parametrize("T", [5, 700])
def test_experts_masked_by_the_bias(low, E, groups, T):
    """Masked experts come last; whole groups of them lose against any other."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe

    per = E // groups
    rng = np.random.default_rng(E)
    x = rng.standard_normal((T, E)).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.05).astype(np.float32)
    bias[::3] = low                     # some of every group
    bias[2 * per:4 * per] = low         # two groups
    for group_top in (1, 2):
        for top_groups in (1, 2, groups - 1):
            K = min(4, per)
            kw = dict(groups=groups, top_groups=top_groups, group_top=group_top)
            want = _order(x, K, "sigmoid", bias, **kw)
            _, ids = moe.route(torch.from_numpy(x).cuda(), K, scores="sigmoid", bias=torch.from_numpy(bias).cuda(), **kw)
            assert np.array_equal(to_host(ids).view(np.int32), want), (group_top, top_groups)


# around the borders of a lone workgroup, of one launch and of two, and pieces that end inside a wave's part
@pytest.mark.parametrize("n", [64, 65, 512, 513, 1024, 1025, 1500, 2049, 4096, 4097, 6145, 20000, 32768, 32769, 70001])
@pytest.mark.parametrize("E", [1, 7, 128, 900, 901, 1024])
def test_dispatch_of_any_number_of_slots(n, E):
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe

    import mx4_util as ref
    rng = np.random.default_rng(n + E)
    ids = rng.integers(-1, E + 1, (n, 1)).astype(np.int32)
    log("dispatch n=%d E=%d" % (n, E))
    for g, want in zip(moe.dispatch(torch.from_numpy(ids).cuda(), E), ref.dispatch(ids, E)):
        assert np.array_equal(to_host(g).view(np.int32), want)


# rows and slots around the ranges that a workgroup counts, and past the sizes that one launch does
@pytest.mark.parametrize("T,K,rows", [(1024, 2, 2047), (1024, 2, 2048), (683, 3, 2049), (1, 1, 5000), (3000, 1, 1), (8191, 8, 65528),
                                      (32768, 8, 262144), (32769, 8, 100), (100, 1, 524289)])
@pytest.mark.parametrize("kind", ["distinct", "dropped"])
def test_combine_gradient_of_any_number_of_rows(T, K, rows, kind):
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe

    H = 8
    log("combine gradient T=%d K=%d rows=%d %s" % (T, K, rows, kind))
    rng = np.random.default_rng(T + rows)
    n = T * K
    position = np.full(n, -1, np.int32)
    named = min(n, rows) if kind == "distinct" else min(n, rows) // 2
    position[rng.permutation(n)[:named]] = rng.permutation(rows)[:named]
    position = position.reshape(T, K)
    y = rng.integers(-4, 5, (rows, H)).astype(np.float32)
    w = rng.integers(-4, 5, (T, K)).astype(np.float32)
    g = rng.integers(-4, 5, (T, H)).astype(np.float32)      # every product and sum is exact
    ty, tw = (torch.from_numpy(a).cuda().requires_grad_() for a in (y, w))
    out = moe.combine(ty, torch.from_numpy(position).cuda(), tw)
    dy, dw = (t.cpu().numpy() for t in torch.autograd.grad(out, (ty, tw), torch.from_numpy(g).cuda()))
    t, k = np.nonzero(position >= 0)
    want_dy, want_dw = np.zeros_like(y), np.zeros_like(w)
    want_dy[position[t, k]] = w[t, k][:, None] * g[t]
    want_dw[t, k] = (y[position[t, k]] * g[t]).sum(1)
    assert np.array_equal(dy, want_dy) and np.array_equal(dw, want_dw)


# rows that several slots name, at sizes where a slot-by-slot search would take seconds
@pytest.mark.parametrize("T,K,rows,H", [(20000, 4, 40000, 8), (20000, 4, 300, 40), (5000, 8, 3, 264), (3000, 5, 7500, 2056)])
def test_combine_gradient_of_many_shared_rows(T, K, rows, H):
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe

    log("combine gradient, shared rows T=%d K=%d rows=%d H=%d" % (T, K, rows, H))
    rng = np.random.default_rng(T + rows)
    position = (rng.permutation(T * K) % rows).reshape(T, K).astype(np.int32)
    y = rng.integers(-4, 5, (rows, H)).astype(np.float32)
    w = rng.integers(-4, 5, (T, K)).astype(np.float32)
    g = rng.integers(-4, 5, (T, H)).astype(np.float32)      # sums of whole numbers below 2^24: exact in any order
    ty, tw = (torch.from_numpy(a).cuda().requires_grad_() for a in (y, w))
    out = moe.combine(ty, torch.from_numpy(position).cuda(), tw)
    dy, dw = (t.cpu().numpy() for t in torch.autograd.grad(out, (ty, tw), torch.from_numpy(g).cuda()))
    want_dy = np.zeros_like(y)
    for k in range(K):
        np.add.at(want_dy, position[:, k], w[:, k:k + 1] * g)
    want_dw = np.stack([(y[position[:, k]] * g).sum(1) for k in range(K)], 1)
    assert np.array_equal(dy, want_dy) and np.array_equal(dw, want_dw)


def test_outputs_of_one_call_are_independent_tensors():
    """They lie in one allocation, but alias nothing and stand on their own."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe, mxfp4

    x = torch.randn((33, 256), device="cuda").bfloat16()
    logits = torch.randn((33, 24), device="cuda")
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            w, ids = moe.route(logits, 3)
            plan = moe.dispatch(ids, 24)
            q = mxfp4.quantize(x, packed=True)
            groups = [(w, ids), tuple(plan), tuple(q.values())]
        for group in groups:
            spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in group)
            assert all(a[1] <= b[0] for a, b in zip(spans, spans[1:]))
            before = [t.clone() for t in group]
            for t in group:
                assert t.is_contiguous() and t.data_ptr() % 256 == 0 and not t._is_view()
                assert t.is_inference() == (mode is torch.inference_mode)
            with mode():
                for i, t in enumerate(group):
                    t.zero_()
                    assert all(torch.equal(a, b) for a, b in list(zip(group, before))[i + 1:])
    w, ids = moe.route(logits, 3)
    leaf = w.requires_grad_()
    (leaf * 2).sum().backward()
    assert torch.equal(leaf.grad, torch.full_like(w, 2.0))
    del w, leaf
    assert int(ids.min()) >= 0        # outlives the others of its call


# the number of slots up to which the gradients' waves count for themselves, and one past it
@pytest.mark.parametrize("T,K,rows,H", [(1024, 1, 1024, 40), (1025, 1, 1025, 40), (113, 9, 1500, 264), (60, 17, 700, 2056), (1024, 1, 7, 8), (3, 64, 100, 33)])
def test_combine_gradient_of_few_slots(T, K, rows, H):
    test_combine_gradient_of_many_shared_rows(T, K, rows, H)
