"""Build libmxfp8.so (gfx950 HIP kernels + C ABI) in-tree with hipcc,
libmxfp8_calib.so, the benchmark's measurement aid (the register-only MFMA
rate; not part of the library), and _mx_torch.so, the extension module of the
tensor-level MXFP4 and mixture-of-experts operators (host C++ against PyTorch's
headers, linked to libmxfp8.so)."""

from __future__ import annotations

import importlib.util
import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libmxfp8.so")
CALIB_PATH = os.path.join(HERE, "libmxfp8_calib.so")
SOURCES = ["api.hip", "quantize.hip", "pack_scales.hip", "gemm.hip", "api_mx4.hip", "mx4_quantize.hip", "mx4_gemm.hip",
           "mx4_gemm_mid.hip", "mx4_gemm_tile.hip", "moe.hip"]
CALIB_SOURCES = ["calib.hip"]
TORCH_PATH = os.path.join(HERE, "_mx_torch.so")
TORCH_SOURCE = "torch_binding.cpp"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

# Packed-FP32 VALU forms are disabled for all device code; hipcc's host pass
# warns that it does not know the feature, which is harmless.
DEVICE_FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
                "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                "-Wall", "-Wno-unused-function", "-Wno-unknown-warning-option"]


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    return None if spec is None else os.path.dirname(spec.origin)


def _host_compile(obj: str, torch_dir: str) -> list:
    """Compile command of the extension module (HIP's headers want the platform named)."""
    inc = os.path.join(torch_dir, "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-isystem", inc,
            "-isystem", os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", "/opt/rocm/include",
            "-I" + sysconfig.get_path("include"), "-c", os.path.join(CSRC, TORCH_SOURCE), "-o", obj]


def _start(cmd):
    """A running compiler, or why there is none."""
    try:
        return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)
    except OSError as e:
        return e


def _succeeded(cmd, p, verbose) -> bool:
    if isinstance(p, OSError):
        sys.stderr.write("FAILED: %s\n%s\n" % (" ".join(cmd), p))
        return False
    out, _ = p.communicate()
    text = "\n".join(line for line in out.decode(errors="replace").splitlines()
                     if "packed-fp32-ops" not in line)
    if p.returncode != 0:
        sys.stderr.write("FAILED: %s\n%s\n" % (" ".join(cmd), text))
    elif verbose and text.strip():
        sys.stderr.write(text + "\n")
    return p.returncode == 0


def _link(cmd, path) -> None:
    tmp = path + ".tmp%d" % os.getpid()
    subprocess.check_call([*cmd, "-o", tmp])
    os.replace(tmp, path)


def build(verbose: bool = False) -> str:
    """Compile and link everything; raises if any part fails.  libmxfp8.so needs
    neither g++ nor PyTorch's headers and is linked without them too."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    procs = []
    objs = []
    for src in SOURCES + CALIB_SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        objs.append(obj)
        cmd = [HIPCC, *DEVICE_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        procs.append((cmd, _start(cmd)))
    binding = os.path.join(BUILD_DIR, TORCH_SOURCE.replace(".cpp", ".o"))
    torch_dir = _torch_dir()
    host = None
    if torch_dir is not None:
        cmd = _host_compile(binding, torch_dir)
        host = (cmd, _start(cmd))
    done = [_succeeded(cmd, p, verbose) for cmd, p in procs]
    host_done = host is not None and _succeeded(*host, verbose)
    if not all(done):
        raise RuntimeError("hipcc compilation failed")
    n = len(SOURCES)
    for path, parts in ((LIB_PATH, objs[:n]), (CALIB_PATH, objs[n:])):
        _link([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", *parts], path)
    if not host_done:
        raise RuntimeError("libmxfp8.so is built, _mx_torch.so is not: " +
                           ("PyTorch was not found" if host is None else "its compilation failed"))
    _link(["g++", "-shared", binding, "-L" + HERE, "-lmxfp8", "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python",
           "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_hip", "-ltorch_hip", "-Wl,-rpath,$ORIGIN"], TORCH_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
