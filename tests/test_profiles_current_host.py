"""The committed profiles' counters are of the present MXFP8 kernels: bench.py
reports them (a change to a kernel's sources calls for new counters)."""

import os

import pytest

import bench

PROFILES = os.path.join(bench.ROOT, "profiles")


def _lines():
    out = []
    for name in sorted(os.listdir(PROFILES)):
        for line in open(os.path.join(PROFILES, name)):
            parts = line.split()
            if parts[:1] == ["traffic"]:
                out.append((parts[1], name))
    return out


def test_there_are_some():
    assert {k for k, _ in _lines()} >= {"gemm:32768x8192x8192", "gemm:8192x14336x4096"}


@pytest.mark.parametrize("key,name", _lines())
def test_profile_is_current(key, name):
    files = bench.GEMM_SOURCES if "gemm" in key.split(":")[0] else bench.QUANTIZE_SOURCES
    assert bench.profiled_traffic(key, files) is not None
