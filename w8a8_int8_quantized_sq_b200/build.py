"""Build the sm_100a CUDA library libsqint8.so in this package directory, and the
Python extension _binding.so that calls it for the mixture-of-experts operators.

One translation unit (csrc/sqint8.cu) holds every kernel and the C ABI of
include/sqint8.h.  Compiled with nvcc for sm_100a only, without fast math,
with the CUDA runtime linked statically; the driver's tensor-map encoder is
looked up at run time, so no libcuda link is needed.
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRC = os.path.join(HERE, "csrc", "sqint8.cu")
LIB = os.path.join(HERE, "libsqint8.so")
BINDING_SRC = os.path.join(HERE, "csrc", "binding.cpp")
BINDING = os.path.join(HERE, "_binding.so")
BINDING_FLAGS = ["-O2", "-std=c++17", "-DNDEBUG", "-shared", "-fPIC"]
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "-shared", "-Xptxas", "-v", "--expt-relaxed-constexpr",
         "-I", os.path.join(ROOT, "include")]


def sources():
    c = os.path.join(HERE, "csrc")
    return [os.path.join(c, f) for f in os.listdir(c) if f != "binding.cpp"] + [
        os.path.join(ROOT, "include", "sqint8.h")]


def _fresh(target: str, inputs) -> bool:
    return os.path.exists(target) and all(
        os.path.getmtime(target) >= os.path.getmtime(s) for s in inputs)


def _run(cmd, what: str, verbose: bool) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError(f"building {what} failed")
    if verbose:
        sys.stderr.write(r.stderr)


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _fresh(LIB, sources()):
        _run([NVCC, *FLAGS, SRC, "-o", LIB + ".tmp"], "libsqint8.so", verbose)
        os.replace(LIB + ".tmp", LIB)
    build_binding(force, verbose)
    return LIB


def binding_key() -> str:
    """What the extension is compiled for: one PyTorch (whose C++ objects it reads and makes),
    one Python, one set of flags.  The file holds it, and one beside it for the next build."""
    import torch
    return "; ".join([f"torch {torch.__version__} {torch.version.git_version}",
                      f"C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                      f"Python {sysconfig.get_config_var('SOABI')}", " ".join(BINDING_FLAGS)])


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """The extension needs PyTorch's headers and libsqint8.so (found beside it at run time)."""
    header = os.path.join(ROOT, "include", "sqint8.h")
    key, key_file = binding_key(), BINDING + ".key"
    if not force and _fresh(BINDING, [BINDING_SRC, header]) and os.path.exists(key_file):
        with open(key_file) as f:
            if f.read() == key:
                return BINDING
    import torch
    from torch.utils import cpp_extension
    lib_dir = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include")
    includes = [*cpp_extension.include_paths(), sysconfig.get_paths()["include"], cuda]
    _run([os.environ.get("CXX", "g++"), *BINDING_FLAGS, f'-DSQ_BINDING_KEY="{key}"',
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[a for i in includes for a in ("-isystem", i)], BINDING_SRC, "-o", BINDING + ".tmp",
          "-L" + HERE, "-l:libsqint8.so", "-L" + lib_dir, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda",
          "-ltorch_python", "-Wl,-rpath,$ORIGIN"], "_binding.so", verbose)
    if os.path.exists(key_file):
        os.remove(key_file)  # never a key beside another build's file
    os.replace(BINDING + ".tmp", BINDING)
    with open(key_file, "w") as f:
        f.write(key)
    return BINDING


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
