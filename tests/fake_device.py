"""The C entry points of csrc/mx4_api.cu over fake_device.cpp: their checks and
choices without a GPU."""
import ctypes
import os
import subprocess
import tempfile

from expert_routed_ffn_gemm_gb300 import binding
from expert_routed_ffn_gemm_gb300 import build as libbuild

HERE = os.path.dirname(os.path.abspath(__file__))
CUDA_INCLUDE = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")


def address(device, at=0, managed=False):
    """16-byte aligned memory of a fake device."""
    return (1 << 44 if managed else 0) | (device + 1) << 40 | (1 << 20) + at


def load():
    libbuild.build(variants=("release",))
    obj = os.path.join(libbuild.VARIANTS["release"][0], "mx4_api.o")
    with tempfile.TemporaryDirectory(prefix="fake_device") as d:
        out = os.path.join(d, "fake.so")
        # -Bsymbolic: the fakes, also where the process has a CUDA runtime loaded
        subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-Wl,-Bsymbolic", "-I", CUDA_INCLUDE,
                        os.path.join(HERE, "fake_device.cpp"), obj, "-o", out], check=True)
        lib = ctypes.CDLL(out)
    real = binding.load()
    for name in binding.EXPORTED:
        if "mx4" in name or "norm" in name:
            f, r = getattr(lib, name), getattr(real, name)
            f.argtypes, f.restype = r.argtypes, r.restype
    return lib


def value(lib, name):
    return ctypes.c_int.in_dll(lib, name).value


def experts(lib, groups, rows, cols, gated=0, device=0):
    """A handle on 4-bit weights of a fake device."""
    lib.cudaSetDevice(device)
    cfg, h = binding.moe_mx4_config(groups, rows, cols, gated), ctypes.c_void_p()
    assert lib.moe_mx4_init(ctypes.byref(cfg), address(device), address(device), ctypes.byref(h)) == binding.MOE_OK
    return h.value
