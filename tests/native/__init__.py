"""Small test libraries, compiled from this folder on the sources of the package."""
import ctypes
import os
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(os.path.dirname(HERE))


def compiled(name: str, folder) -> ctypes.CDLL:
    """``name``.cu of this folder as a library in ``folder``."""
    from trellis_coded_weight_bitshift_b200 import build
    lib = os.path.join(str(folder), f"lib{name}.so")
    cmd = [build._nvcc(), *(f for f in build.NVCC_FLAGS if f not in ("-Xptxas", "-v")), "-I", build.INCLUDE, "-I",
           build.CSRC, "-shared", "-cudart", "static", os.path.join(HERE, f"{name}.cu"), "-o", lib]
    subprocess.run(cmd, check=True, capture_output=True, text=True)
    return ctypes.CDLL(lib)
