"""MXFP4 and mixture-of-experts entry points without a GPU: the headers and the
bindings agree, the headers are C99, and invalid arguments are refused on the
host before anything is launched."""

import ctypes
import os
import re
import shutil
import subprocess

import pytest
import torch

import mxfp8_block_scaled_quantize_amd as mx
from mxfp8_block_scaled_quantize_amd import build as mxbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, NULL, SHAPE, MISALIGNED, FLAGS, WORKSPACE, HIP, LIMIT = range(8)
P = 0x10000   # fake, aligned "device" addresses: never dereferenced


@pytest.fixture(scope="module")
def mods():
    if not os.path.exists(mx.LIB_PATH):
        mxbuild.build()
    from mxfp8_block_scaled_quantize_amd import moe, mxfp4
    return mxfp4, moe


def _header(name):
    return open(os.path.join(ROOT, "include", name)).read()


@pytest.mark.parametrize("header,prefix", [("mxfp4.h", "mxfp4"), ("moe.h", "moe")])
def test_header_and_binding_agree(mods, header, prefix):
    mod = mods[0] if prefix == "mxfp4" else mods[1]
    text = _header(header)
    code = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    names = set(re.findall(r"\b(%s_[a-z0-9_]+)\s*\(" % prefix, code))
    assert names == set(mod.EXPORTED) == set(mod._functions())
    so = ctypes.CDLL(mx.LIB_PATH)
    for n in names:
        getattr(so, n)
        assert callable(getattr(mod, n))
    const = {m.group(1): int(m.group(2)) for m in re.finditer(r"#define (%s_[A-Z0-9_]+) (\d+)u?\b" % prefix.upper(), code)}
    assert const
    bound = {n for n in dir(mod) if re.fullmatch(r"%s_[A-Z0-9_]+" % prefix.upper(), n)}
    assert bound == set(const)
    for n, v in const.items():
        assert getattr(mod, n) == v, n


def test_headers_are_c99(tmp_path):
    cc = shutil.which("gcc")
    if cc is None:
        pytest.skip("no C compiler")
    src = tmp_path / "t.c"
    src.write_text('#include "mxfp4.h"\n#include "moe.h"\n'
                   "int main(void) { return (int)moe_dispatch_workspace_bytes(0, 1, 1); }\n")
    subprocess.check_call([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"), "-c",
                           str(src), "-o", str(tmp_path / "t.o")])


def test_quantize_refusals(mods):
    f = mods[0]._functions()["mxfp4_quantize"]

    def q(x=P, x_rows=64, rows=64, cols=128, ld=128, index=None, flags=1, qr=P, sr=P, qc=P, sc=P):
        return f(x, x_rows, rows, cols, ld, index, flags, qr, sr, qc, sc, None)
    assert q(flags=0) == FLAGS and q(flags=16) == FLAGS and q(flags=5) == FLAGS
    assert q(index=P, flags=3) == FLAGS and q(index=P, flags=2) == FLAGS
    assert q(rows=-1, x_rows=-1) == SHAPE and q(cols=40) == SHAPE and q(ld=120) == SHAPE
    assert q(rows=48, x_rows=48, flags=2) == SHAPE and q(rows=64, flags=18) == SHAPE
    assert q(cols=96, ld=96, flags=17) == SHAPE and q(x_rows=65) == SHAPE
    assert q(x=None) == NULL and q(qr=None) == NULL and q(sr=None) == NULL
    assert q(flags=2, qc=None) == NULL and q(flags=2, sc=None) == NULL
    assert q(x=P + 8) == MISALIGNED and q(ld=132) == MISALIGNED and q(qr=P + 4) == MISALIGNED
    assert q(flags=2, qc=P + 8) == MISALIGNED and q(flags=17, sr=P + 2) == MISALIGNED and q(index=P + 2) == MISALIGNED
    assert q(rows=1 << 41, x_rows=1 << 41) == LIMIT and q(rows=1 << 36, x_rows=1 << 36, cols=32, ld=32) in (LIMIT,)
    assert q(rows=0, x_rows=0, x=None, qr=None, sr=None) == OK and q(cols=0, ld=0, x=None) == OK


def test_dequantize_refusals(mods):
    f = mods[0]._functions()["mxfp4_dequantize"]

    def d(q=P, s=P, rows=4, cols=128, out=P, ld=128, flags=16):
        return f(q, s, rows, cols, out, ld, flags, None)
    assert d(flags=1) == FLAGS and d(cols=96, ld=96) == SHAPE and d(cols=48, flags=0) == SHAPE and d(ld=64) == SHAPE
    assert d(rows=-1) == SHAPE and d(q=None) == NULL and d(s=None) == NULL and d(out=None) == NULL
    assert d(q=P + 8) == MISALIGNED and d(out=P + 8) == MISALIGNED and d(ld=130) == MISALIGNED and d(s=P + 1) == MISALIGNED
    assert d(rows=1 << 41) == LIMIT and d(rows=0, q=None) == OK


def test_gemm_refusals(mods):
    fs = mods[0]._functions()

    def g(a=P, ap=P, b=P, bp=P, c=P, ldc=64, M=4, N=64, K=256, flags=0):
        return fs["mxfp4_gemm"](a, ap, b, bp, c, ldc, M, N, K, flags, None)

    def gg(off=P, G=2, c=P, ldc=64, M=4, N=64, K=256, flags=0):
        return fs["mxfp4_grouped_gemm"](P, P, P, P, off, G, c, ldc, M, N, K, flags, None)
    assert g(flags=2) == FLAGS and g(flags=9) == FLAGS and gg(flags=4) == FLAGS
    assert g(M=-1) == SHAPE and g(N=48) == SHAPE and g(K=64) == SHAPE and g(ldc=32) == SHAPE
    assert g(a=None) == NULL and g(ap=None) == NULL and g(b=None) == NULL and g(bp=None) == NULL and g(c=None) == NULL
    assert g(a=P + 8) == MISALIGNED and g(b=P + 8) == MISALIGNED and g(c=P + 8) == MISALIGNED and g(ldc=68) == MISALIGNED
    assert g(ap=P + 2) == MISALIGNED and g(bp=P + 1) == MISALIGNED
    assert g(K=(1 << 22) + 128) == LIMIT and g(M=1 << 41) == LIMIT and g(N=1 << 31, ldc=1 << 31) == LIMIT
    assert gg(G=0) == SHAPE and gg(G=65536) == SHAPE and gg(off=None) == NULL and gg(off=P + 2) == MISALIGNED
    assert g(M=0, a=None) == OK and g(N=0, ldc=0, c=None) == OK and gg(M=0, off=None) == OK


def test_route_refusals(mods):
    fs = mods[1]._functions()

    def r(x=P, dtype=0, T=4, E=16, ld=16, bias=None, K=2, groups=1, tg=1, gt=2, flags=0, w=P, ids=P):
        return fs["moe_route"](x, dtype, T, E, ld, bias, K, groups, tg, gt, flags, w, ids, None)
    assert r(dtype=3) == FLAGS and r(flags=4) == FLAGS
    assert r(E=0, ld=0) == SHAPE and r(E=1025, ld=1025) == SHAPE and r(ld=15) == SHAPE and r(T=-1) == SHAPE
    assert r(K=0) == SHAPE and r(K=17) == SHAPE and r(E=200, ld=200, K=65) == SHAPE
    assert r(groups=0) == SHAPE and r(groups=3) == SHAPE and r(groups=4, tg=5) == SHAPE and r(groups=4, tg=0) == SHAPE
    assert r(groups=4, tg=1, K=5) == SHAPE and r(groups=4, tg=2, gt=3) == SHAPE and r(groups=128, E=128, ld=128) == SHAPE
    assert r(x=None) == NULL and r(w=None) == NULL and r(ids=None) == NULL
    assert r(x=P + 2) == MISALIGNED and r(x=P + 1, dtype=1) == MISALIGNED and r(bias=P + 2) == MISALIGNED
    assert r(w=P + 2) == MISALIGNED and r(ids=P + 1) == MISALIGNED
    assert r(T=1 << 41) == LIMIT and r(T=1 << 31) == LIMIT and r(T=0, x=None, w=None, ids=None) == OK

    def b(x=P, dtype=0, T=4, E=16, ld=16, ids=P, dw=P, K=2, flags=0, d=P):
        return fs["moe_route_backward"](x, dtype, T, E, ld, ids, dw, K, flags, d, None)
    assert b(dtype=-1) == FLAGS and b(flags=8) == FLAGS and b(K=17) == SHAPE and b(ids=None) == NULL
    assert b(dw=None) == NULL and b(d=None) == NULL and b(d=P + 2) == MISALIGNED and b(T=0, ids=None) == OK


def test_dispatch_refusals(mods):
    moe = mods[1]
    fs = moe._functions()

    def d(ids=P, T=4, E=16, K=2, off=P, tok=P, pos=P, ws=P, n=1 << 24):
        return fs["moe_dispatch"](ids, T, E, K, off, tok, pos, ws, n, None)
    assert d(T=-1) == SHAPE and d(E=0) == SHAPE and d(E=1025) == SHAPE and d(K=0) == SHAPE
    assert d(T=1 << 30, K=2) == LIMIT and d(T=1 << 31, K=1) == LIMIT
    assert d(ids=None) == NULL and d(off=None) == NULL and d(tok=None) == NULL and d(pos=None) == NULL
    assert d(ids=P + 2) == MISALIGNED and d(off=P + 1) == MISALIGNED and d(tok=P + 2) == MISALIGNED and d(pos=P + 2) == MISALIGNED
    need = moe.moe_dispatch_workspace_bytes(100000, 64, 8)
    assert need > 0 and need % (65 * 4) == 0
    assert d(T=100000, E=64, K=8, n=need - 1) == WORKSPACE and d(T=100000, E=64, K=8, ws=None) == WORKSPACE
    assert d(T=100000, E=64, K=8, ws=P + 2) == MISALIGNED
    assert moe.moe_dispatch_workspace_bytes(16, 64, 8) == 0 and moe.moe_dispatch_workspace_bytes(-1, 64, 8) == 0


def test_combine_refusals(mods):
    fs = mods[1]._functions()

    def c(y=P, dtype=1, rows=8, ld=64, pos=P, w=P, T=4, K=2, H=64, out=P):
        return fs["moe_combine"](y, dtype, rows, ld, pos, w, T, K, H, out, None)
    assert c(dtype=7) == FLAGS and c(ld=63) == SHAPE and c(K=0) == SHAPE and c(T=-1) == SHAPE and c(rows=-1) == SHAPE
    assert c(H=-1) == SHAPE and c(y=None) == NULL and c(pos=None) == NULL and c(w=None) == NULL and c(out=None) == NULL
    assert c(y=P + 1) == MISALIGNED and c(out=P + 1) == MISALIGNED and c(pos=P + 2) == MISALIGNED and c(w=P + 2) == MISALIGNED
    assert c(rows=1 << 31) == LIMIT and c(T=1 << 41) == LIMIT and c(T=1 << 37, K=1, rows=1, H=1, ld=1) == LIMIT
    assert c(T=0, pos=None, out=None) == OK and c(H=0, ld=0, out=None) == OK

    def b(y=P, rows=8, ld=64, pos=P, w=P, T=4, K=2, H=64, g=P, ldg=64, dy=P, dw=P, ws=P, n=32):
        return fs["moe_combine_backward"](y, 1, rows, ld, pos, w, T, K, H, g, ldg, dy, dw, ws, n, None)
    assert b(ldg=63) == SHAPE and b(g=None) == NULL and b(pos=None) == NULL and b(ws=None) == WORKSPACE and b(n=31) == WORKSPACE
    assert b(ws=P + 2) == MISALIGNED and b(dy=P + 1) == MISALIGNED and b(dw=P + 2) == MISALIGNED and b(g=P + 1) == MISALIGNED
    assert b(dy=None, dw=None) == OK


def test_helpers_refuse_what_is_not_theirs(mods):
    mxfp4, moe = mods
    cpu = torch.zeros((32, 128), dtype=torch.bfloat16)
    codes, words = torch.zeros((32, 64), dtype=torch.uint8), torch.zeros((1, 32), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        mxfp4.quantize(cpu)
    with pytest.raises(ValueError, match="BF16"):
        mxfp4.quantize(cpu.float())
    with pytest.raises(ValueError, match="BF16"):
        mxfp4.quantize(cpu.t())
    with pytest.raises(ValueError, match="CUDA"):
        mxfp4.dequantize(codes, words)
    with pytest.raises(ValueError, match="CUDA"):
        mxfp4.gemm(codes, words, codes, words)
    with pytest.raises(ValueError, match="even number"):
        mxfp4.gemm(codes, words, codes[:31], words, swiglu=True)
    with pytest.raises(ValueError, match="3-D"):
        mxfp4.grouped_gemm(codes, words, codes, words, words)
    with pytest.raises(ValueError, match="CUDA"):
        moe.route(cpu, 2)
    with pytest.raises(ValueError, match="float32, bfloat16"):
        moe.route(cpu.double(), 2)
    with pytest.raises(ValueError, match="int32"):
        moe.dispatch(words[0], 4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.dispatch(words, 4)
    with pytest.raises(ValueError, match="CUDA"):
        moe.combine(cpu, words, words.float())
    with pytest.raises(ValueError, match="unit column stride"):
        moe.combine(cpu.t(), words, words.float())
