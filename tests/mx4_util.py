"""Plain implementations in 64 bits of the MXFP4 and mixture-of-experts
operators, for the tests (numpy / CPU torch, nothing of the library)."""

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def heavy_bits(shape, seed):
    """BF16 bit patterns of heavy-tailed values, about one in a hundred 32-blocks
    of a row zero."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_t(3, size=shape) * 0.1).astype(np.float32)
    for r, c in zip(rng.integers(0, shape[0], shape[0] // 4 + 1), rng.integers(0, shape[1] // 32 + 1, shape[0] // 4 + 1)):
        x[r, 32 * c:32 * c + 32] = 0
    u = x.view(np.uint32)
    return ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)


def quantize(bits):
    """Codes uint8 [R, C / 2] and scale bytes uint8 [R, C / 32] of BF16 bit patterns [R, C]."""
    r, c = bits.shape
    v = bf16_values(bits).reshape(r, c // 32, 32)
    amax = np.abs(v).max(-1)
    exponent = np.frexp(amax)[1] - 1          # floor(log2 amax) for amax > 0
    x = np.where(amax > 0, np.maximum(exponent - 2, -127), -127)
    mag = np.abs(v) / np.exp2(x.astype(np.float64))[..., None]
    index = np.zeros(mag.shape, np.uint8)
    middle = (E2M1[1:] + E2M1[:-1]) / 2
    for i, m in enumerate(middle):            # a midpoint goes to the even index
        index += ((mag > m) | ((mag == m) & (i % 2 == 1))).astype(np.uint8)
    code = index + 8 * (np.signbit(v)).astype(np.uint8)
    code = code.reshape(r, c // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (x + 127).astype(np.uint8)


def pack(scales):
    """Scale bytes [R, K / 32] -> packed words uint32 [K / 128, R]."""
    r, kb = scales.shape
    b = scales.astype(np.uint32).reshape(r, kb // 4, 4)
    return np.ascontiguousarray((b[..., 0] | b[..., 1] << 8 | b[..., 2] << 16 | b[..., 3] << 24).T)


def dequantize(codes, scales):
    r = codes.shape[0]
    c = np.stack((codes & 15, codes >> 4), -1).reshape(r, -1, 32)
    v = np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]
    return (v * np.exp2(scales.astype(np.float64) - 127)[..., None]).reshape(r, -1)


def random_operand(rng, rows, k):
    """Codes, scale bytes and values of a random operand."""
    codes = rng.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    scales = rng.integers(120, 132, (rows, k // 32), dtype=np.uint8)
    return codes, scales, dequantize(codes, scales)


def route(logits, top_k, scores, bias=None, groups=1, top_groups=1, group_top=2, renormalize=True):
    """weights, ids and the score matrix, in 64 bits."""
    x = np.asarray(logits, np.float64)
    t, e = x.shape
    if scores == "softmax":
        m = x.max(1, keepdims=True)
        p = np.exp(x - np.where(np.isinf(m), 0, m))
        total = p.sum(1, keepdims=True)
        s = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
    else:
        with np.errstate(over="ignore"):
            s = 1 / (1 + np.exp(-x))
    choice = s if bias is None else s + np.asarray(bias, np.float64)
    # without a bias the order is the logits' own (far scores may both round to 0 or 1)
    order_by = x if bias is None else choice
    shut = np.zeros((t, e), bool)
    if groups > 1:
        g = np.sort(choice.reshape(t, groups, -1), -1)[..., ::-1][..., :group_top].sum(-1)
        kept = np.argsort(-g, 1, kind="stable")[:, :top_groups]
        shut = np.ones((t, groups), bool)
        np.put_along_axis(shut, kept, False, 1)
        shut = np.repeat(shut, e // groups, 1)
    ids = np.empty((t, top_k), np.int32)
    for i in range(t):
        ids[i] = sorted(range(e), key=lambda j: (shut[i, j], -order_by[i, j], j))[:top_k]
    w = np.take_along_axis(s, ids, 1)
    if renormalize:
        w = w / (w.sum(1, keepdims=True) + 1e-20)
    return w, ids, s


def route_backward(logits, ids, dw, scores, renormalize):
    x = np.asarray(logits, np.float64)
    s = route(x, 1, scores)[2]
    g = np.zeros_like(s)
    g_chosen = np.asarray(dw, np.float64)
    if renormalize:
        chosen = np.take_along_axis(s, ids, 1)
        total = chosen.sum(1, keepdims=True) + 1e-20
        g_chosen = (g_chosen - (g_chosen * chosen).sum(1, keepdims=True) / total) / total
    np.put_along_axis(g, ids, g_chosen, 1)
    if scores == "softmax":
        return s * (g - (g * s).sum(1, keepdims=True))
    e = np.exp(-np.abs(x))
    return g * e / (1 + e) ** 2


def dispatch(ids, experts):
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < experts)
    bucket = np.where(ok, flat, experts)
    order = np.argsort(bucket, kind="stable")
    n = int(ok.sum())
    position = np.full(flat.size, -1, np.int32)
    position[order[:n]] = np.arange(n, dtype=np.int32)
    token = np.full(flat.size, -1, np.int32)
    token[:n] = order[:n] // ids.shape[1]
    offsets = np.concatenate(([0], np.cumsum(np.bincount(bucket, minlength=experts + 1)[:experts]))).astype(np.int32)
    return offsets, token, position.reshape(ids.shape)


def combine(y, position, weights):
    y, w = np.asarray(y, np.float64), np.asarray(weights, np.float64)
    ok = (position >= 0) & (position < y.shape[0])
    rows = np.where(ok[..., None], y[np.where(ok, position, 0)] if y.shape[0] else 0.0, 0.0)
    return (rows * w[..., None]).sum(1), rows, ok
