"""Key-value cache and rotary entry points without a GPU: headers and bindings
agree, the headers are C99, and invalid arguments are refused on the host before
anything is launched."""

import ctypes
import os
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import kv_util
import mxfp8_block_scaled_quantize_amd as mx
from mxfp8_block_scaled_quantize_amd import build as mxbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, MISALIGNED, FLAGS, WORKSPACE, HIP, LIMIT = range(8)
P = 0x10000   # fake, aligned "device" addresses: never dereferenced


@pytest.fixture(scope="module")
def mods():
    if not os.path.exists(mx.LIB_PATH):
        mxbuild.build()
    from mxfp8_block_scaled_quantize_amd import kvcache, rotary
    return kvcache, rotary


@pytest.mark.parametrize("header,prefix,which", [("kvcache.h", "kv", 0), ("rotary.h", "rotary", 1)])
def test_header_and_binding_agree(mods, header, prefix, which):
    mod = mods[which]
    code = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", header)).read(), flags=re.S)
    names = set(re.findall(r"\b(%s_[a-z0-9_]+)\s*\(" % prefix, code))
    assert names == set(mod.EXPORTED) == set(mod._functions())
    so = ctypes.CDLL(mx.LIB_PATH)
    for n in names:
        getattr(so, n)
        assert callable(getattr(mod, n))
    const = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define (ROTARY_[A-Z0-9_]+) (\d+)u?\b", code)}
    assert {n for n in dir(mod) if n.startswith("ROTARY_")} == set(const)
    for n, v in const.items():
        assert getattr(mod, n) == v, n


def test_headers_are_c99(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "kvcache.h"\n#include "rotary.h"\n'
                   "int main(void) { return (int)kv_attention_workspace_bytes(0, 1, 1, 64, 0, 0, 16, 0, 1, 0); }\n")
    subprocess.check_call([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c",
                           str(src), "-o", str(tmp_path / "t.o")])


def test_extend_refusals(mods):
    f = mods[0]._functions()["kv_extend"]

    def e(table=P, ld=8, width=8, lengths=P, counts=P, requests=4, free=P, count=P, pages=64, page=16, tokens=10, offsets=P,
          out=P, slots=P, positions=P, left=P):
        return f(table, ld, width, lengths, counts, requests, free, count, pages, page, tokens, offsets, out, slots, positions, left,
                 None)
    assert e(page=8) == SHAPE and e(page=24) == SHAPE and e(page=512) == SHAPE and e(page=0) == SHAPE and e(pages=0) == SHAPE
    assert e(ld=7) == SHAPE and e(width=-1) == SHAPE and e(requests=-1) == SHAPE and e(tokens=-1) == SHAPE
    assert e(pages=1 << 28) == LIMIT and e(requests=1 << 24) == LIMIT and e(tokens=(1 << 31) - 1) == LIMIT
    assert e(width=1 << 27, ld=1 << 27) == LIMIT and e(ld=1 << 39) == LIMIT
    for name in ("table", "lengths", "counts", "free", "count", "offsets", "out", "slots", "positions", "left"):
        assert e(**{name: None}) == NULL, name
        assert e(**{name: P + 2}) == MISALIGNED, name


def test_release_refusals(mods):
    f = mods[0]._functions()["kv_release"]

    def r(table=P, ld=8, width=8, lengths=P, finished=P, requests=4, free=P, count=P, pages=64, page=16, out=P, left=P):
        return f(table, ld, width, lengths, finished, requests, free, count, pages, page, out, left, None)
    assert r(page=48) == SHAPE and r(pages=-1) == SHAPE and r(ld=4) == SHAPE and r(requests=-1) == SHAPE
    assert r(pages=1 << 27) == LIMIT and r(requests=1 << 24) == LIMIT
    for name in ("table", "lengths", "finished", "free", "count", "out", "left"):
        assert r(**{name: None}) == NULL, name
    for name in ("table", "lengths", "free", "count", "out", "left"):
        assert r(**{name: P + 1}) == MISALIGNED, name


def test_append_and_read_refusals(mods):
    f, g = mods[0]._functions()["kv_append"], mods[0]._functions()["kv_read"]

    def a(cache=P, pages=4, page=16, heads=2, d=64, k=P, kt=128, kh=64, v=P, vt=128, vh=64, slots=P, tokens=5):
        return f(cache, pages, page, heads, d, k, kt, kh, v, vt, vh, slots, tokens, None)

    def r(cache=P, pages=4, page=16, heads=2, d=64, slots=P, tokens=5, k=P, v=P):
        return g(cache, pages, page, heads, d, slots, tokens, k, v, None)
    for call in (a, r):
        assert call(page=8) == SHAPE and call(pages=0) == SHAPE and call(heads=0) == SHAPE and call(d=96) == SHAPE
        assert call(d=32) == SHAPE and call(tokens=-1) == SHAPE
        assert call(pages=1 << 28) == LIMIT and call(heads=1 << 30) == LIMIT and call(tokens=1 << 33) == LIMIT
        assert call(tokens=(1 << 63) - 1) == LIMIT
        assert call(cache=None) == NULL and call(k=None) == NULL and call(v=None) == NULL and call(slots=None) == NULL
        assert call(cache=P + 8) == MISALIGNED and call(k=P + 8) == MISALIGNED and call(v=P + 2) == MISALIGNED
        assert call(slots=P + 2) == MISALIGNED and call(tokens=0, k=None, v=None, slots=None) == OK
    assert a(kt=-8) == SHAPE and a(vh=-8) == SHAPE and a(kt=12) == MISALIGNED and a(kh=4) == MISALIGNED and a(vt=1) == MISALIGNED


def test_attention_refusals(mods):
    f, ws = mods[0]._functions()["kv_attention"], mods[0]._functions()["kv_attention_workspace_bytes"]

    def t(q=P, qt=512, qh=64, tokens=4, heads=8, cache=P, pages=4, page=16, kv_heads=2, d=64, table=P, ld=8, width=8, lengths=P,
          offsets=None, sequences=4, most=1, scale=0.1, window=0, out=P, lse=P, work=P, bytes_=1 << 40):
        return f(q, qt, qh, tokens, heads, cache, pages, page, kv_heads, d, table, ld, width, lengths, offsets, sequences, most,
                 scale, window, out, lse, work, bytes_, None)
    assert t(tokens=5) == SHAPE and t(heads=7) == SHAPE and t(heads=0) == SHAPE and t(kv_heads=0) == SHAPE and t(d=192) == SHAPE
    assert t(page=4) == SHAPE and t(width=-1) == SHAPE and t(ld=2) == SHAPE and t(most=0) == SHAPE and t(window=-1) == SHAPE
    assert t(tokens=-1, sequences=-1) == SHAPE and t(qt=-8) == SHAPE and t(pages=0) == SHAPE
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        assert t(scale=scale) == SHAPE
    assert t(tokens=1 << 29, sequences=1 << 29) == LIMIT and t(width=1 << 27, ld=1 << 27) == LIMIT
    assert t(heads=1 << 18, kv_heads=2) == LIMIT and t(pages=1 << 28) == LIMIT and t(qt=1 << 39) == LIMIT
    for name in ("q", "cache", "table", "lengths", "out"):
        assert t(**{name: None}) == NULL, name
        assert t(**{name: P + 2}) == MISALIGNED, name
    assert t(lse=P + 2) == MISALIGNED and t(qt=516) == MISALIGNED and t(qh=60) == MISALIGNED and t(offsets=P + 1) == MISALIGNED
    assert t(tokens=0, sequences=0, q=None, out=None) == OK and t(tokens=0, sequences=3, offsets=P, q=None) == OK
    # one long sequence is cut into parts, which meet in the workspace
    sizes = dict(tokens=1, sequences=1, width=4096, ld=4096)
    need = ws(1, 8, 2, 64, 1, 4096, 16, 0, 1, 0)
    assert need > 0 and t(bytes_=need - 1, **sizes) == WORKSPACE and t(work=None, **sizes) == WORKSPACE
    assert t(work=P + 4, **sizes) == MISALIGNED
    assert ws(4, 8, 2, 64, 4, 8, 16, 0, 1, 0) == 0 and ws(4, 7, 2, 64, 4, 4096, 16, 0, 1, 0) == 0


def test_rotary_refusals(mods):
    f = mods[1]._functions()["rotary_rotate"]

    def r(q=P, qt=256, qh=64, qn=4, k=P, kt=128, kh=64, kn=2, dtype=1, tokens=3, d=64, pairs=32, positions=P, turns=P, mag=1.0,
          flags=0, qo=P, ko=P):
        return f(q, qt, qh, qn, k, kt, kh, kn, dtype, tokens, d, pairs, positions, turns, mag, flags, qo, ko, None)
    assert r(dtype=3) == FLAGS and r(dtype=-1) == FLAGS and r(flags=4) == FLAGS
    assert r(pairs=33) == SHAPE and r(pairs=-1) == SHAPE and r(d=0) == SHAPE and r(tokens=-1) == SHAPE and r(qn=-1) == SHAPE
    assert r(kt=-1) == SHAPE and r(d=1 << 17) == LIMIT and r(qn=1 << 21) == LIMIT and r(tokens=1 << 30) == LIMIT
    for name in ("q", "k", "qo", "ko", "positions", "turns"):
        assert r(**{name: None}) == NULL, name
        assert r(**{name: P + 1}) == MISALIGNED, name
    assert r(turns=P + 4) == MISALIGNED and r(dtype=0, q=P + 2) == MISALIGNED
    assert r(tokens=0, q=None) == OK and r(qn=0, kn=0) == OK


def test_tensor_level_refusals_without_a_gpu(mods):
    kvcache, rotary = mods
    cache = kvcache.new(4, 16, 2, 64)
    assert cache.shape == (4, 2, 16 * 68) and cache.dtype == torch.uint8 and int(cache.sum()) == 0
    free, count = kvcache.pool(5)
    assert free.tolist() == [4, 3, 2, 1, 0] and count.tolist() == [5]
    for args in ((4, 8, 2, 64), (4, 16, 2, 96), (0, 16, 2, 64), (4, 16, 0, 64)):
        with pytest.raises(ValueError):
            kvcache.new(*args)
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.append(cache, x, x, i)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.read(cache, i, 64)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.attention(x, cache, torch.zeros((3, 2), dtype=torch.int32), i)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.extend(torch.zeros((3, 2), dtype=torch.int32), i, i, free, count, 4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        kvcache.release(torch.zeros((3, 2), dtype=torch.int32), i, i.bool(), free, count, 16)
    with pytest.raises(ValueError, match="CUDA"):
        rotary.rotate(x, x, i, torch.zeros(32, dtype=torch.float64))
    for call in (lambda: kvcache.append(None, x, x, i), lambda: kvcache.read(cache, None, 64),
                 lambda: kvcache.attention(None, cache, i, i), lambda: rotary.rotate(None, None, i, i)):
        with pytest.raises(TypeError):
            call()


def test_turns(mods):
    rotary = mods[1]
    n, base, trained = 32, 10000.0, 4096
    plain = base ** (-np.arange(n) / n) / (2 * np.pi)
    t, m = rotary.turns(64)
    assert t.dtype == torch.float64 and m == 1.0 and np.allclose(t.numpy(), plain, rtol=1e-14)
    assert np.allclose(rotary.turns(64, scaling="linear", factor=4.0)[0].numpy(), plain / 4, rtol=1e-14)
    ntk = rotary.turns(64, scaling="ntk", factor=4.0)[0].numpy()
    assert np.isclose(ntk[0], plain[0]) and np.isclose(ntk[-1], plain[-1] / 4)
    for scaling in ("yarn", "bands"):
        t, m = rotary.turns(64, scaling=scaling, factor=8.0, trained=trained)
        ratio = plain / t.numpy()
        rounds = plain * trained
        assert np.all(np.diff(ratio) >= -1e-12) and np.isclose(ratio[0], 1) and np.isclose(ratio[-1], 8)
        assert np.isclose(m, 0.1 * np.log(8.0) + 1 if scaling == "yarn" else 1.0)
        high, low = (32.0, 1.0) if scaling == "yarn" else (4.0, 1.0)
        # a pair's border is rounded outwards to whole pairs: one pair off at most
        step = base ** (1 / n)
        assert np.allclose(ratio[rounds >= high * step], 1) and np.allclose(ratio[rounds <= low / step], 8)
    assert np.allclose(rotary.turns(64, scaling="bands", factor=1.0, trained=trained)[0].numpy(), plain)
    for bad in (dict(dims=63), dict(dims=0), dict(dims=64, base=1.0), dict(dims=64, factor=0.5), dict(dims=64, scaling="other"),
                dict(dims=64, scaling="yarn"), dict(dims=2, scaling="ntk"), dict(dims=64, scaling="bands", trained=8, high=1.0)):
        with pytest.raises(ValueError):
            rotary.turns(**bad)


def test_layer_refusals():
    from mxfp8_block_scaled_quantize_amd.attention_layer import MXFP4Attention
    for bad in ((96, 4, 2, 64), (128, 1, 1, 64), (128, 4, 3, 64), (128, 4, 2, 32)):
        with pytest.raises(ValueError):
            MXFP4Attention(*bad)
    layer = MXFP4Attention(128, 4, 2, 64)
    with pytest.raises(ValueError, match="input"):
        layer(torch.zeros((3, 128)), None, None, None)


def test_plain_forms():
    """The plain forms against each other: the cache's bytes and their values."""
    rng = np.random.default_rng(0)
    bits = rng.integers(0x3E00, 0x4100, (2, 3, 2, 16, 64)).astype(np.uint16)
    cache = torch.from_numpy(kv_util.cache_bytes(bits[0], bits[1]))
    k, v = kv_util.cache_values(cache, 16, 64)
    x = kv_util.mx4_util.bf16_values(bits)
    assert np.abs(k.numpy() - x[0]).max() <= x.max() / 4 and np.abs(v.numpy() - x[1]).max() <= x.max() / 4
    assert not np.array_equal(k.numpy(), v.numpy())
