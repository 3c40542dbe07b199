"""The variant that a product of given sizes takes, asked of the library's own
rule: csrc/linear_plan.h, compiled alone with g++."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "selective_state_space_mssm_amd", "csrc")
PATHS = ["rows", "columns", "tile128", "tile256"]
DTYPES = {"f32": 0, "bf16": 1, "f8": 2}
SOURCE = r"""
#include "linear_plan.h"
extern "C" void plan(int64_t M, int64_t K, int64_t N, int dtype, int out, int64_t cus, int64_t* r) {
    const mssm::LinearPlan p = mssm::plan_linear(M, K, N, dtype, out, cus);
    r[0] = static_cast<int64_t>(p.path); r[1] = p.full; r[2] = p.rest; r[3] = p.splits; r[4] = static_cast<int64_t>(p.ws_bytes);
}
extern "C" void grid(int64_t groups, int64_t* r) {
    const mssm::LinearGrid g = mssm::linear_grid(groups);
    r[0] = g.x; r[1] = g.y;
}
"""


@functools.lru_cache(maxsize=1)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I", os.path.join(ROOT, "include"),
                        "-I", CSRC, src, "-o", so], check=True)
        lib = ctypes.CDLL(so)
    lib.plan.argtypes = [ctypes.c_int64] * 3 + [ctypes.c_int] * 2 + [ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    lib.grid.argtypes = [ctypes.c_int64, ctypes.POINTER(ctypes.c_int64)]
    lib.plan.restype = lib.grid.restype = None
    return lib


def plan(M, K, N, dtype, out, cus=256):
    """(path, whole tiles, cut tiles, parts of each of these, workspace bytes)"""
    r = (ctypes.c_int64 * 5)()
    _lib().plan(M, K, N, DTYPES[dtype], DTYPES[out], cus, r)
    return (PATHS[r[0]], *r[1:])


def grid(groups):
    """(x, y) of the tile kernel's grid for so many workgroups"""
    r = (ctypes.c_int64 * 2)()
    _lib().grid(groups, r)
    return r[0], r[1]
