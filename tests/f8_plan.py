"""The library's choice of e4m3 kernel (csrc/f8_plan.h), built for the host."""

import ctypes
import os
import subprocess

from bitlinear_w1_a8_amd import build

SOURCE = """
#include "f8_plan.h"
extern "C" int plan(int64_t t, int64_t n, int64_t k, int bf16, int cus) {
  return bl::f8_kernel(t, n, k, bf16, cus);
}
extern "C" int rows(int64_t t, int64_t n, int cus) { return bl::f8_few_rows(t, n, cus); }
"""

KERNELS = ("few1", "few2", "small", "tall", "square", "wide", "turns")


def compiled(folder):
    """f8_kernel(T, N, K, bfloat16 outputs, CUs) -> its name, and f8_few_rows(T, N, CUs), from a
    library built in `folder`."""
    src, lib = os.path.join(folder, "plan.cpp"), os.path.join(folder, "plan.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", build.CSRC, src, "-o", lib], check=True)
    built = ctypes.CDLL(lib)
    fn, rows = built.plan, built.rows
    rows.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]
    fn.argtypes = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_int]
    return lambda t, n, k, bf16, cus: KERNELS[fn(t, n, k, int(bf16), cus)], rows
