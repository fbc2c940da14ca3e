"""Builds tests/packed_host.cu (host code alone runs) and loads it."""
import ctypes
import os
import subprocess
import tempfile

from exact_attention_20_gb300 import build as fa_build

_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "packed_host.cu")
        with tempfile.TemporaryDirectory() as tmp:
            out = os.path.join(tmp, "packed_host.so")
            subprocess.run([fa_build.nvcc(), *fa_build.COMPILE_FLAGS, "-shared", "-cudart", "static",
                            "-I", os.path.join(fa_build.ROOT, "include"), "-I", os.path.join(fa_build.PKG, "csrc"),
                            "-o", out, src], check=True)
            _lib = ctypes.CDLL(out)
    return _lib
