"""Tensors past 2^32 bytes and 2^31 elements: sampled rows on both sides of the
border against the plain implementation in 64 bits."""

import numpy as np
import pytest

import mx4_util as ref
from gpu_util import bf16_to_f64, log, need_gpu, to_dev, to_host

pytestmark = [pytest.mark.gpu, pytest.mark.slow]

ROWS, COLS = 300032, 8192          # 2.46e9 elements, 4.9 GB of BF16
BORDER = 2 ** 31 // COLS           # the row that holds element 2^31
SAMPLE = [0, 1, 777, BORDER - 1, BORDER, BORDER + 1, ROWS - 130, ROWS - 1]


def _big(torch):
    # a row times a factor of its own: cheap to make, different everywhere
    g = torch.Generator(device="cuda").manual_seed(0)
    x = torch.randn((1, COLS), generator=g, device="cuda").bfloat16()
    return x * torch.randn((ROWS, 1), generator=g, device="cuda").bfloat16()


def test_quantize_and_dequantize():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    x = _big(torch)
    log("quantize %d x %d" % (ROWS, COLS))
    q = mxfp4.quantize(x, rowwise=True, colwise=True, packed=True)
    at = torch.tensor(SAMPLE, device="cuda")
    codes, scales = ref.quantize(to_host(x[at]))
    assert np.array_equal(to_host(q["q_row"][at]), codes)
    assert np.array_equal(to_host(q["p_row"][:, at].contiguous()), ref.pack(scales))
    cols = torch.tensor([0, 5, COLS - 1], device="cuda")
    codes, scales_t = ref.quantize(to_host(x[:, cols].t().contiguous()))
    assert np.array_equal(to_host(q["q_colT"][cols]), codes)
    assert np.array_equal(to_host(q["p_colT"][:, cols].contiguous()), ref.pack(scales_t))
    index = at.to(torch.int32)
    g = mxfp4.quantize(x, packed=True, index=index)
    assert torch.equal(g["q_row"], q["q_row"][at]) and torch.equal(g["p_row"], q["p_row"][:, at])
    del x, g
    y = mxfp4.dequantize(q["q_row"], q["p_row"])
    got = bf16_to_f64(to_host(y[at]))
    codes = to_host(q["q_row"][at])
    assert np.array_equal(got, ref.dequantize(codes, scales))


def test_gemm_output():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    rng = np.random.default_rng(1)
    K = 128
    b, sb, vb = ref.random_operand(rng, COLS, K)
    a = torch.randint(0, 256, (ROWS, K // 2), dtype=torch.uint8, device="cuda")
    words = torch.full((1, ROWS), 0x7F7E7D80, dtype=torch.int32, device="cuda")
    log("gemm %d x %d" % (ROWS, COLS))
    c = mxfp4.gemm(a, words, to_dev(b), to_dev(ref.pack(sb).view(np.int32)))
    at = torch.tensor(SAMPLE, device="cuda")
    va = ref.dequantize(to_host(a[at]), np.tile(np.array([0x80, 0x7D, 0x7E, 0x7F], np.uint8), (len(SAMPLE), 1)))
    want, err = va @ vb.T, K * 2.0 ** -24 * (np.abs(va) @ np.abs(vb).T)
    got = bf16_to_f64(to_host(c[at]))
    assert np.all(np.abs(got - want) <= err + 2.0 ** -8 * (np.abs(want) + err))


@pytest.mark.parametrize("rows", [3, 700])
def test_grouped_gemm_experts(rows):
    """Experts past byte 2^32 of B, with few rows each and with many."""
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    G, N, K = 66, 16384, 8192                       # 4.4 GB of codes
    M = G * rows
    b = torch.randint(0, 256, (G, N, K // 2), dtype=torch.uint8, device="cuda")
    a = torch.randint(0, 256, (M, K // 2), dtype=torch.uint8, device="cuda")
    pa = torch.full((K // 128, M), 0x7F7F7F7F, dtype=torch.int32, device="cuda")
    pb = torch.full((K // 128, G * N), 0x7F7F7F7F, dtype=torch.int32, device="cuda")
    off = torch.arange(0, M + 1, rows, dtype=torch.int32, device="cuda")
    log("grouped gemm of %d rows each" % rows)
    c = mxfp4.grouped_gemm(a, pa, b, pb, off)
    cols = torch.tensor([0, 1000, N - 1], device="cuda")
    for g in (0, 31, 63, 64, G - 1):
        r = torch.tensor([g * rows, g * rows + rows - 1], device="cuda")
        ones = np.full((2, K // 32), 127, np.uint8)
        va = ref.dequantize(to_host(a[r]), ones)
        vb = ref.dequantize(to_host(b[g][cols]), np.full((3, K // 32), 127, np.uint8))
        want, err = va @ vb.T, K * 2.0 ** -24 * (np.abs(va) @ np.abs(vb).T)
        got = bf16_to_f64(to_host(c[r][:, cols].contiguous()))
        assert np.all(np.abs(got - want) <= err + 2.0 ** -8 * (np.abs(want) + err)), g


def test_combine_and_gradients():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import moe
    y = _big(torch).requires_grad_()
    pos = torch.tensor([SAMPLE, SAMPLE[::-1][:7] + [-1]], dtype=torch.int32, device="cuda")
    # the second token names seven of the first one's rows again: those are sums
    w = torch.randn(2, 8, device="cuda").requires_grad_()
    d = torch.randn(2, COLS, device="cuda").bfloat16()
    log("combine from %d x %d" % (ROWS, COLS))
    out = moe.combine(y, pos, w)
    dy, dw = torch.autograd.grad(out, (y, w), d)
    at = torch.tensor(SAMPLE, device="cuda")
    rows = bf16_to_f64(to_host(y.detach()[at]))
    ww, dd = w.detach().double().cpu().numpy(), d.double().cpu().numpy()
    second = rows[::-1][:7]
    want = np.stack((ww[0] @ rows, ww[1, :7] @ second))
    mags = np.stack((np.abs(ww[0]) @ np.abs(rows), np.abs(ww[1, :7]) @ np.abs(second)))
    err = 9 * 2.0 ** -24 * mags
    assert np.all(np.abs(out.detach().double().cpu().numpy() - want) <= err + 2.0 ** -8 * (np.abs(want) + err))
    want_dw = np.stack((rows @ dd[0], np.append(second @ dd[1], 0.0)))
    mags = np.stack((np.abs(rows) @ np.abs(dd[0]), np.append(np.abs(second) @ np.abs(dd[1]), 0.0)))
    assert np.all(np.abs(dw.double().cpu().numpy() - want_dw) <= (COLS + 2) * 2.0 ** -24 * mags)
    want_dy = ww[0][:, None] * dd[0]
    mags = np.abs(want_dy)
    for k in range(7):
        want_dy[7 - k] += ww[1, k] * dd[1]
        mags[7 - k] += np.abs(ww[1, k] * dd[1])
    err = 3 * 2.0 ** -24 * mags
    assert np.all(np.abs(bf16_to_f64(to_host(dy[at])) - want_dy) <= err + 2.0 ** -8 * (np.abs(want_dy) + err))
    dy[at] = 0
    assert int(torch.count_nonzero(dy.view(torch.int32))) == 0
