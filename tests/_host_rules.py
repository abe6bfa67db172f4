"""The kernels' CUDA-free rules (csrc headers), compiled for the host."""
import ctypes
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def build(include=None) -> ctypes.CDLL:
    """tests/native/host_rules.cpp against the headers in `include`."""
    include = include or os.path.join(ROOT, "paged_kv_cache_274_gb300", "csrc")
    with tempfile.TemporaryDirectory() as tmp:
        lib = os.path.join(tmp, "libhost_rules.so")
        subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-Wno-unknown-pragmas", "-fPIC", "-shared", "-I", include, "-o", lib,
                        os.path.join(ROOT, "tests", "native", "host_rules.cpp")], check=True)
        return ctypes.CDLL(lib)
