"""The library's host side (zero_api.hip) built with g++ over host_double.cpp:
argument checks, dispatch and bookkeeping on a machine without a GPU."""
from __future__ import annotations

import ctypes
import os
import shutil
import subprocess

import zero_partitioned_optimizer_flatten_amd as zero
from zero_partitioned_optimizer_flatten_amd import build as zb

TESTS = os.path.dirname(os.path.abspath(__file__))
ROCM = os.path.dirname(os.path.dirname(zb.HIPCC))
FLAGS = ["-std=c++17", "-O1", "-g", "-shared", "-fPIC", "-fstack-protector-all", "-w",
         "-D__HIP_PLATFORM_AMD__", "-D__align__(n)=__attribute__((aligned(n)))",
         "-DHIP_SYMBOL(x)=(x)", "-I" + os.path.join(ROCM, "include"), "-I" + zb.CSRC]


def available() -> bool:
    return bool(shutil.which("g++")) and os.path.exists(
        os.path.join(ROCM, "include", "hip", "hip_runtime_api.h"))


def build(out_dir: str) -> str:
    so = os.path.join(out_dir, "libzero_host.so")
    subprocess.check_call(["g++", *FLAGS, "-x", "c++", os.path.join(zb.CSRC, "zero_api.hip"),
                           os.path.join(TESTS, "host_double.cpp"), "-o", so])
    return so


def load(path: str):
    """The functions with the signatures of the package's own library."""
    was, zero._lib, zero.LIB_PATH = (zero._lib, zero.LIB_PATH), None, path
    try:
        L = zero.lib()
    finally:
        zero._lib, zero.LIB_PATH = was
    L.hipMalloc.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
    return L


class Host:
    """The loaded library with the few calls the tests make of it."""

    def __init__(self, path: str):
        self.L = load(path)

    def malloc(self, nbytes: int) -> int:
        p = ctypes.c_void_p()
        assert self.L.hipMalloc(ctypes.byref(p), max(1, nbytes)) == 0
        return p.value

    def adamw(self, shapes, world=1, rank=0, bits=32):
        """Context of 2-d shapes (rows, row elements)."""
        h = ctypes.c_void_p()
        n = len(shapes)
        d = (ctypes.c_int64 * n)(*[s[0] for s in shapes])
        r = (ctypes.c_int64 * n)(*[s[1] for s in shapes])
        rc = self.L.zero_adamw_init(n, d, r, world, rank, 1e-3, 0.9, 0.95, 1e-8, bits, 1,
                                    ctypes.byref(h))
        assert rc == zero.ZERO_OK, self.error()
        return h

    def pointers(self, ptrs):
        return (ctypes.c_void_p * len(ptrs))(*ptrs)

    def error(self) -> str:
        return self.L.zero_last_error().decode()
