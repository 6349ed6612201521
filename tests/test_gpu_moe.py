"""Expert routing, dispatch and combination against plain implementations in
64 bits."""

import numpy as np
import pytest

import mx4_util as ref
from gpu_util import log, need_gpu, to_dev, to_host

pytestmark = pytest.mark.gpu


def _moe():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    return torch, moe


def _half_step(torch, dtype):
    return torch.finfo(dtype).eps / 2


# tokens, experts, top_k, scores, bias, groups, top_groups, group_top, renormalize, dtype
ROUTES = [
    (1, 1, 1, "softmax", False, 1, 1, 1, True, "float32"),
    (1, 8, 2, "softmax", False, 1, 1, 1, True, "bfloat16"),
    (5, 60, 6, "sigmoid", False, 1, 1, 1, False, "float16"),
    (37, 64, 8, "softmax", True, 1, 1, 1, True, "bfloat16"),
    (130, 128, 8, "softmax", False, 1, 1, 1, True, "bfloat16"),
    (130, 128, 8, "softmax", False, 1, 1, 1, False, "float32"),
    (67, 127, 7, "sigmoid", True, 1, 1, 1, True, "float32"),
    (33, 160, 6, "softmax", False, 8, 3, 1, False, "float32"),
    (33, 160, 6, "softmax", False, 8, 3, 2, False, "bfloat16"),
    (129, 256, 8, "sigmoid", True, 8, 4, 2, True, "float32"),
    (64, 256, 8, "sigmoid", False, 8, 4, 2, True, "bfloat16"),
    (20, 300, 12, "sigmoid", True, 4, 2, 1, True, "float16"),
    (20, 384, 8, "softmax", True, 6, 5, 2, True, "bfloat16"),
    (9, 513, 64, "softmax", True, 1, 1, 1, True, "float32"),
    (9, 1024, 33, "sigmoid", True, 64, 7, 2, True, "float32"),
    (6, 12, 12, "softmax", False, 4, 4, 2, True, "float32"),
    (6, 24, 6, "sigmoid", False, 24, 6, 2, True, "float32"),      # groups of one expert
]


def _logits(torch, T, E, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((T, E), generator=g).to(getattr(torch, dtype))


@pytest.mark.parametrize("case", ROUTES, ids=[str(i) for i in range(len(ROUTES))])
@pytest.mark.parametrize("pad", [0, 3])
def test_route_and_gradient(case, pad):
    torch, moe = _moe()
    T, E, K, scores, with_bias, groups, top_groups, group_top, renorm, dtype = case
    log("route %s pad=%d" % (case, pad))
    whole = _logits(torch, T, E + pad, dtype, E + K)
    x = whole[:, :E]
    bias = torch.randn(E, generator=torch.Generator().manual_seed(1)) * 0.05 if with_bias else None
    kw = dict(scores=scores, groups=groups, top_groups=top_groups, group_top=group_top, renormalize=renorm)
    want_w, want_ids, _ = ref.route(x.double().numpy(), K, bias=None if bias is None else bias.numpy(), **kw)
    dev = whole.cuda().requires_grad_()
    w, ids = moe.route(dev[:, :E], K, bias=None if bias is None else bias.cuda(), **kw)
    assert np.array_equal(to_host(ids).view(np.int32), want_ids)
    # some ten fp32 operations, each within an ulp or two (2^-23)
    assert np.all(np.abs(w.detach().cpu().double().numpy() - want_w) <= 16 * 2.0 ** -23 * want_w + 1e-37)
    dw = torch.randn((T, K), generator=torch.Generator().manual_seed(2))
    got = torch.autograd.grad(w, dev, dw.cuda())[0].cpu().double().numpy()
    want = ref.route_backward(x.double().numpy(), want_ids, dw.numpy(), scores, renorm)
    # sums of K products of scores and dw: relative to the largest of the row
    size = np.abs(want).max(1, keepdims=True) + (np.abs(dw.numpy()) * want_w).max(1, keepdims=True)
    tol = _half_step(torch, x.dtype) * np.abs(want) + 64 * 2.0 ** -23 * size
    if x.dtype == torch.float16:
        tol = tol + 2.0 ** -25   # half a subnormal step
    assert np.all(np.abs(got[:, :E] - want) <= tol)
    assert np.all(got[:, E:] == 0)


def test_route_gradient_against_differences():
    torch, moe = _moe()
    for scores, renorm in (("softmax", True), ("softmax", False), ("sigmoid", True), ("sigmoid", False)):
        T, E, K = 16, 48, 4
        g = torch.Generator().manual_seed(11)
        # top experts well apart, so that a step changes no choice
        x = torch.stack([torch.randperm(E, generator=g) for _ in range(T)]).float() * 0.1
        v = torch.randn((T, E), generator=g) * 0.3
        dw = torch.randn((T, K), generator=g)
        leaf = x.cuda().requires_grad_()
        w, ids = moe.route(leaf, K, scores=scores, renormalize=renorm)
        d = torch.autograd.grad(w, leaf, dw.cuda())[0].cpu().double()
        h = 2.0 ** -7
        side = []
        for s in (h, -h):
            ws, i = moe.route((x + s * v).cuda(), K, scores=scores, renormalize=renorm)
            assert torch.equal(i, ids)
            side.append((ws.cpu().double() * dw.double()).sum(1))
        slope = (side[0] - side[1]) / (2 * h)
        # third derivatives of products of scores: h^2 |v|^3 of the weights' size; fp32 noise 1e-6 / h
        size = (dw.abs().double() * w.detach().cpu().double()).sum(1)
        limit = 8 * (h * 1.5) ** 2 * size + 4e-6 / h * size
        assert torch.all(((d * v.double()).sum(1) - slope).abs() <= limit), (scores, renorm)


def test_route_orders_scores_closer_than_32_bits():
    torch, moe = _moe()
    T, E, K = 64, 96, 8
    rng = np.random.default_rng(0)
    bias = np.full(E, 0.05, np.float32)
    for i in rng.permutation(E):
        bias[i] = np.float32(0.05) + np.float32(2.0 ** -28) * np.float32(rng.integers(0, 40))
    x = np.zeros((T, E), np.float32)          # scores 0.5: the sums differ in the 64-bit digits alone
    _, want, _ = ref.route(x, K, "sigmoid", bias=bias)
    _, ids = moe.route(to_dev(x), K, scores="sigmoid", bias=to_dev(bias))
    assert np.array_equal(to_host(ids).view(np.int32), want)
    # and groups whose sums do
    _, want, _ = ref.route(x, K, "sigmoid", bias=bias, groups=12, top_groups=5, group_top=2)
    _, ids = moe.route(to_dev(x), K, scores="sigmoid", bias=to_dev(bias), groups=12, top_groups=5, group_top=2)
    assert np.array_equal(to_host(ids).view(np.int32), want)


def test_route_many_rows_with_bias():
    """Enough rows that some have choices within the 32-bit error."""
    torch, moe = _moe()
    T, E, K = 3000, 256, 8
    x = _logits(torch, T, E, "bfloat16", 3)
    bias = (torch.randn(E, generator=torch.Generator().manual_seed(4)) * 0.05)
    _, want, _ = ref.route(x.double().numpy(), K, "sigmoid", bias=bias.numpy(), groups=8, top_groups=4)
    _, ids = moe.route(x.cuda(), K, scores="sigmoid", bias=bias.cuda(), groups=8, top_groups=4)
    assert np.array_equal(to_host(ids).view(np.int32), want)


def test_route_masks_ties_and_infinities():
    torch, moe = _moe()
    inf, low = float("inf"), torch.finfo(torch.float32).min
    x = torch.zeros((7, 40))
    x[1] = -inf                                   # nothing left
    x[2, 3:] = -inf                               # fewer than top_k left
    x[3] = low                                    # the lowest value everywhere
    x[4, ::2] = low
    x[5] = float("nan")
    x[6, 7] = inf
    for scores in ("softmax", "sigmoid"):
        w, ids = moe.route(x.cuda(), 5, scores=scores)
        w, ids = w.cpu(), ids.cpu()
        for row in ids.tolist():
            assert len(set(row)) == 5 and all(0 <= e < 40 for e in row)
        for r in (0, 1, 3):
            assert ids[r].tolist() == [0, 1, 2, 3, 4]
        assert ids[2].tolist() == [0, 1, 2, 3, 4]
        assert ids[4].tolist() == [1, 3, 5, 7, 9]
        assert ids[6, 0] == 7
        assert torch.all(w[1] == 0)
        assert torch.allclose(w[0], torch.full((5,), 0.2), rtol=1e-6)
        assert torch.allclose(w[2, :3], torch.full((3,), 1 / 3.), rtol=1e-6) and torch.all(w[2, 3:] == 0)
        assert torch.allclose(w[4], torch.full((5,), 0.2), rtol=1e-6)
        if scores == "softmax":
            assert torch.allclose(w[3], torch.full((5,), 0.2), rtol=1e-6)
            assert torch.isnan(w[6]).all()
        else:
            assert torch.all(w[3] == 0)
        assert torch.isnan(w[5]).all()
    # +0 and -0 are the same logit
    z = torch.zeros((1, 10))
    z[0, ::2] = -0.0
    assert moe.route(z.cuda(), 4)[1].tolist() == [[0, 1, 2, 3]]
    # experts that a bias of -inf takes out come last, behind them closed groups
    b = torch.zeros(40)
    b[:36] = -inf
    assert moe.route(x[:1].cuda(), 5, scores="sigmoid", bias=b.cuda())[1].tolist() == [[36, 37, 38, 39, 0]]
    d = x[1:2].cuda().requires_grad_()
    w, _ = moe.route(d, 5)
    assert torch.all(torch.autograd.grad(w.sum(), d)[0] == 0)


def test_route_gradient_without_use_and_of_expanded_weights():
    torch, moe = _moe()
    x = _logits(torch, 10, 32, "float32", 0).cuda().requires_grad_()
    w, ids = moe.route(x, 4, renormalize=False)
    assert not ids.requires_grad
    got = torch.autograd.grad(w.sum(), x)[0].cpu().double().numpy()        # an expanded gradient of ones
    want = ref.route_backward(x.detach().cpu().numpy(), to_host(ids).view(np.int32), np.ones((10, 4)), "softmax", False)
    assert np.all(np.abs(got - want) <= 64 * 2.0 ** -23)


DISPATCHES = [(0, 4, 2), (1, 1, 1), (1, 4, 4), (16, 256, 8), (63, 3, 2), (511, 5, 8), (512, 60, 8), (513, 384, 8), (1000, 64, 5),
              (4099, 128, 8), (3000, 1024, 3), (40000, 17, 4)]


@pytest.mark.parametrize("T,E,K", DISPATCHES)
@pytest.mark.parametrize("outside", [False, True])
def test_dispatch(T, E, K, outside):
    torch, moe = _moe()
    rng = np.random.default_rng(T + E + K)
    # a few popular experts, some without a slot
    ids = np.minimum((rng.random((T, K)) ** 3 * E).astype(np.int32), E - 1)
    if outside and T:
        ids[rng.random((T, K)) < 0.2] = -1
        ids[rng.random((T, K)) < 0.1] = E
        ids.reshape(-1)[0] = 2 ** 31 - 1
        ids.reshape(-1)[-1] = -2 ** 31
    log("dispatch T=%d E=%d K=%d outside=%s" % (T, E, K, outside))
    got = moe.dispatch(to_dev(ids), E)
    for g, want, name in zip(got, ref.dispatch(ids, E), got._fields):
        assert np.array_equal(to_host(g).view(np.int32), want), name


def test_dispatch_all_to_one_expert():
    torch, moe = _moe()
    ids = np.full((5000, 4), 6, np.int32)
    for g, want in zip(moe.dispatch(to_dev(ids), 9), ref.dispatch(ids, 9)):
        assert np.array_equal(to_host(g).view(np.int32), want)


# tokens, rows, top_k, hidden
COMBINES = [(1, 1, 1, 1), (3, 24, 8, 256), (16, 128, 8, 4096), (5, 12, 2, 100), (70, 700, 9, 264), (33, 99, 3, 1000),
            (129, 258, 2, 2056), (40, 700, 17, 512), (7, 20, 2, 2049), (1025, 8200, 8, 64), (2050, 5000, 5, 72)]


@pytest.mark.parametrize("T,rows,K,H", COMBINES)
@pytest.mark.parametrize("dtype", ["bfloat16", "float16", "float32"])
@pytest.mark.parametrize("kind", ["distinct", "dropped", "shared"])
def test_combine_and_gradients(T, rows, K, H, dtype, kind):
    torch, moe = _moe()
    rng = np.random.default_rng(T + rows + K + H)
    tt = getattr(torch, dtype)
    if kind == "shared":       # several slots name one row
        pos = rng.integers(0, max(1, rows // 3), (T, K)).astype(np.int32)
    else:
        pos = np.resize(rng.permutation(max(rows, T * K))[:T * K], (T, K)).astype(np.int32)   # past the rows: dropped
        if kind == "dropped":
            pos[rng.random((T, K)) < 0.3] = -1
    y = torch.from_numpy(rng.standard_normal((rows, H))).to(tt)
    w = torch.from_numpy(rng.standard_normal((T, K))).float()
    d = torch.from_numpy(rng.standard_normal((T, H))).to(tt)
    log("combine T=%d rows=%d K=%d H=%d %s %s" % (T, rows, K, H, dtype, kind))
    yd, wd = y.cuda().requires_grad_(), w.cuda().requires_grad_()
    out = moe.combine(yd, to_dev(pos), wd)
    with torch.no_grad():
        assert torch.equal(moe.combine(yd, to_dev(pos), wd), out)
    half, u = _half_step(torch, tt), 2.0 ** -24
    tiny = 2.0 ** -25 if tt == torch.float16 else 0.0
    yy, ww, dd = y.double().numpy(), w.double().numpy(), d.double().numpy()
    want, rowsv, ok = ref.combine(yy, pos, ww)
    err = (K + 1) * u * (np.abs(rowsv) * np.abs(ww)[..., None]).sum(1)
    assert np.all(np.abs(out.detach().cpu().double().numpy() - want) <= half * (np.abs(want) + err) + err + tiny)
    dy, dw = torch.autograd.grad(out, (yd, wd), d.cuda())
    want_dw = np.where(ok, (rowsv * dd[:, None]).sum(-1), 0.0)
    assert np.all(np.abs(dw.cpu().double().numpy() - want_dw) <= (H + 2) * u * (np.abs(rowsv) * np.abs(dd)[:, None]).sum(-1))
    want_dy, mag, n = np.zeros_like(yy), np.zeros_like(yy), 0
    for t in range(T):
        for k in range(K):
            if ok[t, k]:
                want_dy[pos[t, k]] += ww[t, k] * dd[t]
                mag[pos[t, k]] += np.abs(ww[t, k] * dd[t])
    n = np.bincount(pos[ok].reshape(-1), minlength=rows)[:, None]
    err = (n + 1) * u * mag
    got = dy.cpu().double().numpy()
    assert np.all(np.abs(got - want_dy) <= half * (np.abs(want_dy) + err) + err + tiny)
    assert np.all(got[n[:, 0] == 0] == 0)


def test_combine_strides_single_gradients_and_expanded_gradients():
    torch, moe = _moe()
    g = torch.Generator().manual_seed(0)
    base = torch.randn((30, 300), generator=g).bfloat16().cuda()
    pos = torch.randperm(30, generator=g)[:24].to(torch.int32).view(8, 3).cuda()
    w = torch.rand((8, 3), generator=g).cuda()
    y = base[:, 4:260]                       # rows that start at 8 bytes
    want = moe.combine(y.contiguous(), pos, w)
    assert torch.equal(moe.combine(y, pos, w), want)
    for leaf_y, leaf_w in ((True, False), (False, True)):
        yl, wl = y.detach().clone().requires_grad_(leaf_y), w.clone().requires_grad_(leaf_w)
        out = moe.combine(yl, pos, wl)
        out.backward(torch.ones((1, 1), dtype=out.dtype, device="cuda").expand(8, 256))
        both_y, both_w = y.detach().clone().requires_grad_(), w.clone().requires_grad_()
        moe.combine(both_y, pos, both_w).backward(torch.ones_like(want))
        if leaf_y:
            assert torch.equal(yl.grad, both_y.grad) and wl.grad is None
        else:
            assert torch.equal(wl.grad, both_w.grad) and yl.grad is None


def test_combine_gradient_against_differences():
    torch, moe = _moe()
    g = torch.Generator().manual_seed(5)
    T, K, H = 12, 4, 96
    y = torch.randn((T * K, H), generator=g).cuda()
    w = torch.rand((T, K), generator=g).cuda()
    pos = torch.randperm(T * K, generator=g).to(torch.int32).view(T, K).cuda()
    d = torch.randn((T, H), generator=g).cuda()
    vy, vw = torch.randn((T * K, H), generator=g).cuda(), torch.randn((T, K), generator=g).cuda()
    yl, wl = y.clone().requires_grad_(), w.clone().requires_grad_()
    gy, gw = torch.autograd.grad(moe.combine(yl, pos, wl), (yl, wl), d)
    h = 2.0 ** -6
    up, down = (moe.combine(y + s * vy, pos, w + s * vw).double() for s in (h, -h))
    slope = ((up - down) * d.double()).sum() / (2 * h)     # the function is bilinear: differences are exact
    want = (gy.double() * vy.double()).sum() + (gw.double() * vw.double()).sum()
    size = (up.abs() * d.abs().double()).sum()
    assert abs(float(slope - want)) <= 16 * 2.0 ** -24 / h * float(size)


def test_a_layer_in_mxfp4():
    """route, dispatch, gathered quantize, grouped SwiGLU product, quantize,
    grouped product, combine: every step on the results of the one before."""
    torch, moe = _moe()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    T, H, F, E, K = 77, 512, 256, 16, 4
    g = torch.Generator().manual_seed(6)
    x = torch.randn((T, H), generator=g).bfloat16().cuda()
    logits = torch.randn((T, E), generator=g).cuda()
    up = (torch.randn((E * 2 * F, H), generator=g) * 0.05).bfloat16().cuda()
    down = (torch.randn((E * H, F), generator=g) * 0.05).bfloat16().cuda()
    qu, qd = mxfp4.quantize(up, packed=True), mxfp4.quantize(down, packed=True)
    weights, ids = moe.route(logits, K)
    plan = moe.dispatch(ids, E)
    qx = mxfp4.quantize(x, packed=True, index=plan.token)
    h = mxfp4.grouped_gemm(qx["q_row"], qx["p_row"], qu["q_row"].view(E, 2 * F, H // 2), qu["p_row"], plan.offsets, swiglu=True)
    qh = mxfp4.quantize(h, packed=True)
    y = mxfp4.grouped_gemm(qh["q_row"], qh["p_row"], qd["q_row"].view(E, H, F // 2), qd["p_row"], plan.offsets)
    out = moe.combine(y, plan.position, weights)
    values = {n: mxfp4.dequantize(q["q_row"], q["p_row"]).double().cpu() for n, q in (("x", qx), ("u", qu), ("h", qh), ("d", qd))}
    token, off = plan.token.cpu().long(), plan.offsets.cpu().tolist()
    codes, scales = ref.quantize(to_host(x)[token.numpy()])
    assert np.array_equal(to_host(qx["q_row"]), codes)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        gate, u2 = (values["x"][r] @ values["u"].view(E, 2 * F, H)[e].T).chunk(2, 1)
        want = torch.nn.functional.silu(gate) * u2
        assert torch.all((h[r].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + H * 2.0 ** -22 * (want.abs() + 1))
        want = values["h"][r] @ values["d"].view(E, H, F)[e].T
        assert torch.all((y[r].double().cpu() - want).abs() <= 2.0 ** -8 * want.abs() + F * 2.0 ** -22 * (want.abs() + 1))
    want, _, _ = ref.combine(y.double().cpu().numpy(), to_host(plan.position).view(np.int32), weights.double().cpu().numpy())
    assert np.all(np.abs(out.double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want) + 1e-5)
