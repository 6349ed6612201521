"""The build without g++ or without PyTorch: libmxfp8.so needs neither and is
linked, and the missing extension module is an error.  The compilers are
stand-ins that leave an empty output file."""

import os
import sys

import pytest

from mxfp8_block_scaled_quantize_amd import build as mxbuild

COMPILER = """#!%s
import sys
open(sys.argv[sys.argv.index("-o") + 1], "w").close()
sys.exit(%d)
"""


def _compiler(path, status=0):
    path.write_text(COMPILER % (sys.executable, status))
    path.chmod(0o755)


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build into an empty folder, with a PATH of its own."""
    tools = tmp_path / "tools"
    tools.mkdir()
    _compiler(tmp_path / "hipcc")
    monkeypatch.setattr(mxbuild, "HIPCC", str(tmp_path / "hipcc"))
    monkeypatch.setenv("PATH", str(tools))
    monkeypatch.setattr(mxbuild, "BUILD_DIR", str(tmp_path / "_build"))
    for name in ("LIB_PATH", "CALIB_PATH", "TORCH_PATH"):
        monkeypatch.setattr(mxbuild, name, str(tmp_path / os.path.basename(getattr(mxbuild, name))))
    return tmp_path


def _built(tree):
    return {p.name for p in tree.iterdir() if p.suffix == ".so"}


def test_everything(tree):
    _compiler(tree / "tools" / "g++")
    assert mxbuild.build() == mxbuild.LIB_PATH
    assert _built(tree) == {"libmxfp8.so", "libmxfp8_calib.so", "_mx_torch.so"}


def test_without_a_host_compiler(tree):
    with pytest.raises(RuntimeError, match="_mx_torch.so is not"):
        mxbuild.build()
    assert _built(tree) == {"libmxfp8.so", "libmxfp8_calib.so"}


def test_host_compiler_fails(tree):
    _compiler(tree / "tools" / "g++", status=1)
    with pytest.raises(RuntimeError, match="_mx_torch.so is not"):
        mxbuild.build()
    assert _built(tree) == {"libmxfp8.so", "libmxfp8_calib.so"}


def test_without_pytorch(tree, monkeypatch):
    _compiler(tree / "tools" / "g++")
    monkeypatch.setattr(mxbuild.importlib.util, "find_spec", lambda name: None)
    with pytest.raises(RuntimeError, match="PyTorch was not found"):
        mxbuild.build()
    assert _built(tree) == {"libmxfp8.so", "libmxfp8_calib.so"}


def test_device_compiler_fails(tree):
    _compiler(tree / "hipcc", status=1)
    _compiler(tree / "tools" / "g++")
    with pytest.raises(RuntimeError, match="hipcc compilation failed"):
        mxbuild.build()
    assert _built(tree) == set()
