"""MXFP4 quantize, dequantize and products against the plain implementation in
64 bits."""

import numpy as np
import pytest

import mx4_util as ref
from gpu_util import bf16_to_f64, log, need_gpu, to_dev, to_dev_bf16, to_host

pytestmark = pytest.mark.gpu


def _mxfp4():
    torch = need_gpu()
    from mxfp8_block_scaled_quantize_amd import mxfp4
    return torch, mxfp4


def _words(a):
    return to_dev(a.view(np.int32))


def _every_pattern():
    """Rows of one amax exponent each, whose other values are every BF16 pattern
    of the five exponents from it down, with both signs."""
    rows = []
    for e in range(255):
        top = (e << 7) | 0x7F
        lo = max(0, e - 4) << 7
        near = np.arange(lo, top + 1, dtype=np.uint16)
        near = np.concatenate((near, near | 0x8000))
        near = np.resize(near, -(-near.size // 31) * 31).reshape(-1, 31)
        block = np.concatenate((np.full((near.shape[0], 1), top, np.uint16), near), 1).reshape(-1)
        rows.append(np.resize(block, 32 * 44))
    return np.stack(rows)


def test_quantize_every_bf16_pattern_under_every_scale():
    torch, mxfp4 = _mxfp4()
    bits = _every_pattern()
    log("mxfp4 quantize of %s" % (bits.shape,))
    got = mxfp4.quantize(to_dev_bf16(bits), packed=True)
    codes, scales = ref.quantize(bits)
    assert np.array_equal(to_host(got["p_row"]), ref.pack(scales))
    assert np.array_equal(to_host(got["q_row"]), codes)


def test_dequantize_every_code_under_every_scale():
    torch, mxfp4 = _mxfp4()
    codes = np.tile((np.arange(16, dtype=np.uint8) * 17), (254, 2)).reshape(254, 32)[:, :16]
    codes = np.concatenate((codes, codes[:, ::-1], codes ^ 0x50, codes ^ 0x0A), 1)     # [254, 64]: 4 blocks
    scales = np.repeat(np.arange(254, dtype=np.uint8)[:, None], 4, 1)
    want = ref.dequantize(codes, scales)
    for s in (to_dev(scales), _words(ref.pack(scales))):
        got = bf16_to_f64(to_host(mxfp4.dequantize(to_dev(codes), s)))
        # E2M1 value times a power of two: exact in BF16 up to its largest value
        fits = np.abs(want) < 2.0 ** 128
        assert np.array_equal(got[fits], want[fits])
        assert np.all(np.isinf(got[~fits]) & (np.sign(got[~fits]) == np.sign(want[~fits])))
    zero = to_host(mxfp4.dequantize(to_dev(codes), to_dev(scales)))[want == 0]
    assert set(np.unique(zero)) == {0, 0x8000}


@pytest.mark.parametrize("R,C,ld", [(1, 32, 32), (1, 128, 128), (3, 96, 104), (33, 640, 640), (130, 1056, 1064), (32, 4096, 4096),
                                    (257, 512, 512), (4100, 2080, 2080)])
@pytest.mark.parametrize("packed", [False, True])
def test_quantize_rowwise(R, C, ld, packed):
    torch, mxfp4 = _mxfp4()
    if packed and C % 128:
        C += 128 - C % 128
        ld = max(ld, C)
    bits = ref.heavy_bits((R, ld), R + C)
    log("mxfp4 rowwise R=%d C=%d ld=%d packed=%s" % (R, C, ld, packed))
    got = mxfp4.quantize(to_dev_bf16(bits)[:, :C], packed=packed)
    codes, scales = ref.quantize(bits[:, :C])
    assert np.array_equal(to_host(got["q_row"]), codes)
    if packed:
        assert np.array_equal(to_host(got["p_row"]), ref.pack(scales))
    else:
        assert np.array_equal(to_host(got["s_row"]), scales)


@pytest.mark.parametrize("R,C", [(32, 32), (128, 128), (160, 96), (384, 640), (1024, 416), (512, 1152)])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("rowwise", [False, True])
def test_quantize_colwise(R, C, packed, rowwise):
    torch, mxfp4 = _mxfp4()
    if packed:
        R, C = -(-R // 128) * 128, -(-C // 128) * 128 if rowwise else C
    bits = ref.heavy_bits((R, C), R * 3 + C)
    log("mxfp4 colwise R=%d C=%d packed=%s rowwise=%s" % (R, C, packed, rowwise))
    got = mxfp4.quantize(to_dev_bf16(bits), rowwise=rowwise, colwise=True, packed=packed)
    for name, b in (("row", bits), ("colT", np.ascontiguousarray(bits.T)))[0 if rowwise else 1:]:
        codes, scales = ref.quantize(b)
        assert np.array_equal(to_host(got["q_" + name]), codes), name
        if packed:
            assert np.array_equal(to_host(got["p_" + name]), ref.pack(scales)), name
        else:
            assert np.array_equal(to_host(got["s_" + name]), scales), name


def test_quantize_gathered_rows():
    torch, mxfp4 = _mxfp4()
    bits = ref.heavy_bits((50, 384), 5)
    index = np.array([3, 3, -1, 49, 50, 0, 7, 2 ** 31 - 1, -2 ** 31, 12, 48] * 7, np.int32)
    ok = (index >= 0) & (index < 50)
    gathered = np.where(ok[:, None], bits[np.where(ok, index, 0)], np.uint16(0))
    codes, scales = ref.quantize(gathered)
    for packed in (False, True):
        got = mxfp4.quantize(to_dev_bf16(bits), packed=packed, index=to_dev(index))
        assert np.array_equal(to_host(got["q_row"]), codes)
        want = ref.pack(scales) if packed else scales
        assert np.array_equal(to_host(got["p_row" if packed else "s_row"]), want)


def test_empty_inputs():
    torch, mxfp4 = _mxfp4()
    z = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    got = mxfp4.quantize(z, packed=True)
    assert got["q_row"].shape == (0, 128) and got["p_row"].shape == (2, 0)
    assert mxfp4.dequantize(got["q_row"], got["p_row"]).shape == (0, 256)
    b = mxfp4.quantize(torch.ones((64, 256), dtype=torch.bfloat16, device="cuda"), packed=True)
    assert mxfp4.gemm(got["q_row"], got["p_row"], b["q_row"], b["p_row"]).shape == (0, 64)
    # no reduction: zeros, or the old values with accumulate
    a0 = torch.empty((5, 0), dtype=torch.uint8, device="cuda")
    b0 = torch.empty((64, 0), dtype=torch.uint8, device="cuda")
    pa, pb = (torch.empty((0, n), dtype=torch.int32, device="cuda") for n in (5, 64))
    out = torch.full((5, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(mxfp4.gemm(a0, pa, b0, pb, out=out, accumulate=True), torch.full_like(out, 3.0))
    assert torch.equal(mxfp4.gemm(a0, pa, b0, pb, out=out), torch.zeros_like(out))


# The fp32 sum of K products is within K 2^-24 of the sum of their magnitudes
# whatever the order; the BF16 rounding adds 2^-8 of the value.
def _bounds(x, y):
    want = x @ y.T
    return want, x.shape[1] * 2.0 ** -24 * (np.abs(x) @ np.abs(y).T)


def _swiglu(gate, up):
    (g, dg), (u, du) = gate, up
    with np.errstate(over="ignore"):
        s = g / (1 + np.exp(-g))
    # |SiLU'| <= 1.1; silu_f32 is within 1.14 (4 + |g|) 2^-23 of its value
    return s * u, 1.1 * dg * (np.abs(u) + du) + np.abs(s) * du + 1.14 * (4 + np.abs(g)) * 2.0 ** -23 * np.abs(s * u)


def _close(got, want, err, label):
    tol = err + 2.0 ** -8 * (np.abs(want) + err)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), "%s: %d off, first at %s: %g for %g (tol %g)" % (
        label, bad.sum(), np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])


SHAPES = [(1, 32, 128), (1, 1024, 4096), (3, 96, 384), (16, 64, 640), (17, 160, 256), (37, 32, 1152), (64, 256, 2048),
          (65, 288, 512), (100, 1024, 1280), (129, 544, 896), (255, 256, 256), (300, 800, 640), (513, 1056, 384),
          (1000, 2080, 768), (2049, 1312, 512)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_gemm(M, N, K, mode):
    torch, mxfp4 = _mxfp4()
    rng = np.random.default_rng(M * 7 + N * 3 + K)
    a, sa, va = ref.random_operand(rng, M, K)
    b, sb, vb = ref.random_operand(rng, N * (2 if mode == "swiglu" else 1), K)
    if mode == "swiglu":   # gates of a few units
        sa, va = sa - 3, va / 8
        sb, vb = sb - 3, vb / 8
    log("mxfp4 gemm M=%d N=%d K=%d %s" % (M, N, K, mode))
    args = (to_dev(a), _words(ref.pack(sa)), to_dev(b), _words(ref.pack(sb)))
    want, err = _bounds(va, vb)
    if mode == "accumulate":
        old = ref.heavy_bits((M, N + 8), 3)
        out = to_dev_bf16(old)
        got = to_host(mxfp4.gemm(*args, out=out[:, :N], accumulate=True))
        assert np.array_equal(to_host(out)[:, N:], old[:, N:])
        o = bf16_to_f64(old[:, :N])
        want, err = want + o, err + 2.0 ** -24 * (np.abs(want) + np.abs(o))
    else:
        got = to_host(mxfp4.gemm(*args, swiglu=mode == "swiglu"))
        if mode == "swiglu":
            want, err = _swiglu((want[:, :N], err[:, :N]), (want[:, N:], err[:, N:]))
    _close(bf16_to_f64(got), want, err, "M=%d N=%d K=%d %s" % (M, N, K, mode))


# Enough tiles for the larger ones: 64 x 128, 128 x 128 and 256 x 256, with ends
# inside a tile, half steps of K and a single one.
LARGE = [(1100, 2080, 256), (1300, 3104, 384), (2100, 2080, 640), (3000, 4128, 128), (4000, 2080, 384)]


@pytest.mark.parametrize("M,N,K", LARGE)
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_gemm_of_many_tiles(M, N, K, mode):
    test_gemm(M, N, K, mode)


def test_gemm_is_the_same_for_every_tile_choice():
    """Rows of a product do not depend on how many rows there are: the codes'
    products and 32-element sums are exact, only their fp32 order differs."""
    torch, mxfp4 = _mxfp4()
    rng = np.random.default_rng(12)
    N, K = 1056, 2048
    a, sa, va = ref.random_operand(rng, 3000, K)
    b, sb, vb = ref.random_operand(rng, N, K)
    want, err = _bounds(va, vb)
    bd, pb = to_dev(b), _words(ref.pack(sb))
    for M in (1, 15, 16, 31, 33, 64, 127, 200, 255, 257, 640, 1111, 3000):
        log("mxfp4 gemm of the first %d rows" % M)
        got = mxfp4.gemm(to_dev(a[:M]), _words(ref.pack(sa[:M])), bd, pb)
        _close(bf16_to_f64(to_host(got)), want[:M], err[:M], "M=%d" % M)


COUNTS = [[5], [0, 0, 7, 0], [1, 0, 16, 17, 33, 0, 2, 64], [300, 0, 1, 257, 40], [0] * 65 + [3] + [0] * 4 + [130, 1],
          [700, 600, 0, 513]]


@pytest.mark.parametrize("counts", COUNTS, ids=[str(i) for i in range(len(COUNTS))])
@pytest.mark.parametrize("N,K", [(64, 256), (288, 640)])
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_grouped_gemm(counts, N, K, mode):
    torch, mxfp4 = _mxfp4()
    G, M = len(counts), sum(counts) + 3           # three rows outside every group
    rng = np.random.default_rng(M + N + K)
    rows = N * (2 if mode == "swiglu" else 1)
    a, sa, va = ref.random_operand(rng, M, K)
    b, sb, vb = ref.random_operand(rng, G * rows, K)
    if mode == "swiglu":
        sa, va, sb, vb = sa - 3, va / 8, sb - 3, vb / 8
    offsets = np.concatenate(([0], np.cumsum(counts))).astype(np.int32)
    old = ref.heavy_bits((M, N), 9)
    out = to_dev_bf16(old)
    log("mxfp4 grouped %s N=%d K=%d %s" % (counts[:8], N, K, mode))
    got = mxfp4.grouped_gemm(to_dev(a), _words(ref.pack(sa)), to_dev(b.reshape(G, rows, K // 2)), _words(ref.pack(sb)),
                             to_dev(offsets), out=out, accumulate=mode == "accumulate", swiglu=mode == "swiglu")
    got = to_host(got)
    assert np.array_equal(got[M - 3:], old[M - 3:])
    for g in range(G):
        r = slice(offsets[g], offsets[g + 1])
        want, err = _bounds(va[r], vb[g * rows:(g + 1) * rows])
        if mode == "accumulate":
            o = bf16_to_f64(old[r])
            want, err = want + o, err + 2.0 ** -24 * (np.abs(want) + np.abs(o))
        if mode == "swiglu":
            want, err = _swiglu((want[:, :N], err[:, :N]), (want[:, N:], err[:, N:]))
        _close(bf16_to_f64(got[r]), want, err, "group %d" % g)


@pytest.mark.parametrize("counts,N,K", [([2500, 0, 1, 1900, 300, 505], 2080, 384), ([5000, 200], 4128, 128), ([17] * 39 + [40], 1056, 384),
                                        ([0, 4100, 0, 0, 4700, 1], 2080, 384), ([1500, 1003], 1600, 640)],
                         ids=["6", "2", "40", "6empty", "2b"])
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_grouped_gemm_of_many_tiles(counts, N, K, mode):
    test_grouped_gemm(counts, N, K, mode)


def test_grouped_gemm_with_one_group_of_nearly_all_rows():
    """The choice of kernel goes by the average; the rows may all be one expert's."""
    test_grouped_gemm([0] * 20 + [900] + [0] * 10 + [1], 288, 640, "plain")
    test_grouped_gemm([0] * 3 + [700] + [0] * 60, 96, 384, "swiglu")


def test_grouped_gemm_invalid_offsets_stay_inside():
    """Bounds are clamped into [0, M] and raised to the largest one before."""
    torch, mxfp4 = _mxfp4()
    M, N, K, G = 70, 64, 256, 5
    rng = np.random.default_rng(4)
    a, sa, va = ref.random_operand(rng, M, K)
    b, sb, vb = ref.random_operand(rng, G * N, K)
    offsets = np.array([-7, 20, 4, 1000, 60, 2 ** 31 - 1], np.int32)
    edges = np.maximum.accumulate(np.clip(offsets, 0, M))
    old = ref.heavy_bits((M, N), 2)
    got = bf16_to_f64(to_host(mxfp4.grouped_gemm(to_dev(a), _words(ref.pack(sa)), to_dev(b.reshape(G, N, K // 2)),
                                                 _words(ref.pack(sb)), to_dev(offsets), out=to_dev_bf16(old))))
    for g in range(G):
        r = slice(edges[g], edges[g + 1])
        _close(got[r], *_bounds(va[r], vb[g * N:(g + 1) * N]), "group %d" % g)


def test_grouped_gemm_invalid_offsets_with_many_rows():
    torch, mxfp4 = _mxfp4()
    for M, N, K, G in ((3000, 1056, 384, 6), (9000, 2080, 384, 6), (700, 96, 256, 6)):
        rng = np.random.default_rng(M)
        a, sa, va = ref.random_operand(rng, M, K)
        b, sb, vb = ref.random_operand(rng, G * N, K)
        offsets = np.array([-2 ** 31, M // 3, M // 5, M // 2, 2 ** 31 - 1, 7, -1], np.int32)
        edges = np.maximum.accumulate(np.clip(offsets, 0, M))
        log("mxfp4 grouped, offsets %s" % offsets)
        got = bf16_to_f64(to_host(mxfp4.grouped_gemm(to_dev(a), _words(ref.pack(sa)), to_dev(b.reshape(G, N, K // 2)),
                                                     _words(ref.pack(sb)), to_dev(offsets))))
        for g in range(G):
            r = slice(edges[g], edges[g + 1])
            _close(got[r], *_bounds(va[r], vb[g * N:(g + 1) * N]), "group %d" % g)


def test_overlapping_rows_are_refused():
    torch, mxfp4 = _mxfp4()
    import mxfp8_block_scaled_quantize_amd as mx
    from mxfp8_block_scaled_quantize_amd import moe
    one = torch.ones((1, 256), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mx.MXFP8Error, match="SHAPE"):
        mxfp4.quantize(one.expand(64, 256))
    with pytest.raises(mx.MXFP8Error, match="SHAPE"):
        moe.route(one.expand(64, 256), 4)
    position = torch.zeros((2, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(mx.MXFP8Error, match="SHAPE"):
        moe.combine(one.expand(64, 256), position, position.float())
    # one row has no stride to speak of
    odd = torch.ones((3, 300), dtype=torch.bfloat16, device="cuda").as_strided((1, 256), (3, 1))
    assert torch.equal(mxfp4.quantize(odd)["q_row"], mxfp4.quantize(one)["q_row"])


def test_infinities_and_nan_do_not_fault():
    torch, mxfp4 = _mxfp4()
    x = torch.randn((64, 256), device="cuda").bfloat16()
    x[1, 3], x[2, 40], x[3] = float("inf"), float("nan"), float("-inf")
    q = mxfp4.quantize(x, colwise=False, packed=True)
    clean = torch.tensor([r for r in range(64) if r not in (1, 2, 3)], device="cuda")
    want = mxfp4.quantize(x[clean], packed=True)
    assert torch.equal(q["q_row"][clean], want["q_row"]) and torch.equal(q["p_row"][:, clean], want["p_row"])


def test_gemm_extreme_scales():
    """Scale bytes over the whole range: sums past BF16's range are infinite,
    the others keep their tolerance."""
    torch, mxfp4 = _mxfp4()
    rng = np.random.default_rng(8)
    M, N, K = 40, 64, 256
    a, sa, _ = ref.random_operand(rng, M, K)
    b, sb, _ = ref.random_operand(rng, N, K)
    sa = np.repeat(rng.integers(60, 250, (M, 1), dtype=np.uint8), K // 32, 1)
    sb = np.repeat(rng.integers(60, 140, (N, 1), dtype=np.uint8), K // 32, 1)
    va, vb = ref.dequantize(a, sa), ref.dequantize(b, sb)
    got = bf16_to_f64(to_host(mxfp4.gemm(to_dev(a), _words(ref.pack(sa)), to_dev(b), _words(ref.pack(sb)))))
    want, err = _bounds(va, vb)
    mags = np.abs(va) @ np.abs(vb).T
    fits = (mags < 2.0 ** 127) & (mags > 2.0 ** -100)
    assert fits.any()
    _close(got[fits], want[fits], err[fits], "extreme scales")


def test_round_trip_of_a_linear_layer_in_mxfp4():
    """quantize -> gemm -> quantize -> gemm on a stream of its own, against the
    values that codes and scales stand for."""
    torch, mxfp4 = _mxfp4()
    x, w = (torch.randn(n, 512, device="cuda").bfloat16() for n in (200, 384))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    qx, qw = (mxfp4.quantize(t, packed=True, stream=side) for t in (x, w))
    y = mxfp4.gemm(qx["q_row"], qx["p_row"], qw["q_row"], qw["p_row"], stream=side)
    vx, vw = (mxfp4.dequantize(q["q_row"], q["p_row"], stream=side) for q in (qx, qw))
    side.synchronize()
    vx, vw = (bf16_to_f64(to_host(t)) for t in (vx, vw))
    _close(bf16_to_f64(to_host(y)), *_bounds(vx, vw), "linear layer")


# more groups than rows: workgroups only for the groups that can have rows
@pytest.mark.parametrize("counts", [[0] * 63 + [1], [1] + [0] * 200, [0, 2, 0, 0, 1, 0, 0, 0, 1], [0] * 64 + [3] + [0] * 30 + [1, 1] + [0] * 60,
                                    [1] * 5 + [0] * 90 + [1] * 20, [0, 0, 0]],
                         ids=["last", "first", "few", "over64", "ones", "none"])
@pytest.mark.parametrize("N,K", [(64, 256), (288, 640)])
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_grouped_gemm_of_more_groups_than_rows(counts, N, K, mode):
    test_grouped_gemm(counts, N, K, mode)


def test_grouped_gemm_invalid_offsets_of_more_groups_than_rows():
    torch, mxfp4 = _mxfp4()
    M, N, K = 3, 64, 256
    for offsets in ([-7, 2, 1, 1000, 60, 2 ** 31 - 1], [5, 4, 3, 2, 1, 0], [-1, -2 ** 31, 0, 1, -5, 2], [2, 0, 0, 0, 0, 0, 3]):
        offsets = np.array(offsets, np.int32)
        G = len(offsets) - 1
        rng = np.random.default_rng(4)
        a, sa, va = ref.random_operand(rng, M, K)
        b, sb, vb = ref.random_operand(rng, G * N, K)
        edges = np.maximum.accumulate(np.clip(offsets, 0, M))
        old = ref.heavy_bits((M, N), 2)
        log("mxfp4 grouped, offsets %s" % offsets)
        bits = to_host(mxfp4.grouped_gemm(to_dev(a), _words(ref.pack(sa)), to_dev(b.reshape(G, N, K // 2)),
                                          _words(ref.pack(sb)), to_dev(offsets), out=to_dev_bf16(old)))
        got = bf16_to_f64(bits)
        outside = np.ones(M, bool)
        for g in range(G):
            r = slice(edges[g], edges[g + 1])
            outside[r] = False
            _close(got[r], *_bounds(va[r], vb[g * N:(g + 1) * N]), "group %d" % g)
        assert np.array_equal(bits[outside], old[outside])


# Sizes that the other lists leave without some tile: few rows in blocks of 32
# and of 16, 64 x 64, 64 x 128, 128 x 128 and 256 x 256, with and without half
# steps of K, ends of groups inside tiles.
@pytest.mark.parametrize("M,N,K", [(40, 3104, 256), (40, 1600, 128), (200, 1312, 128), (300, 5152, 1920), (2900, 4128, 256),
                                   (2900, 2080, 128), (2900, 4128, 128), (1500, 1312, 384)])
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_gemm_of_other_tiles(M, N, K, mode):
    test_gemm(M, N, K, mode)


@pytest.mark.parametrize("counts,N,K", [([1500, 298], 96, 256), ([1] * 7 + [0, 5] * 11 + [0], 288, 1920), ([12, 0, 3] * 8 + [1, 0, 4, 2, 0, 0], 4128, 640),
                                        ([4000, 1998], 4128, 1920), ([1701, 2296], 5152, 1152), ([2, 0, 0, 30, 9, 96] * 5, 1056, 256)],
                         ids=["2", "30", "30wide", "2large", "2larger", "30uneven"])
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_grouped_gemm_of_other_tiles(counts, N, K, mode):
    test_grouped_gemm(counts, N, K, mode)


# few rows, workgroups of 16 columns (long K) and the sizes next to it
@pytest.mark.parametrize("M,N,K", [(1, 32, 4224), (5, 288, 7168), (33, 1056, 6272), (29, 1024, 8192), (16, 4096, 4224), (17, 4128, 4224)])
@pytest.mark.parametrize("mode", ["plain", "accumulate", "swiglu"])
def test_gemm_of_few_rows_and_long_k(M, N, K, mode):
    test_gemm(M, N, K, mode)
